// Root-mean-square norm with the residual's addition, the residual stream kept
// in 8 bits, and the backward pass from either form.
//
//   h = x + residual (rounded to the storage type)    rstd = 1 / sqrt(mean h^2 + eps)
//   y = h rstd gain
//   kept: for 128 consecutive elements of a row, scale = max|h| / 448 and
//         code = e4m3(h 448 / max|h|); n = code scale rstd stands for h rstd
//   backward, n the normalised row:  dn = dy gain,
//         dx = rstd (dn - n mean(dn n)) + upstream,  dgain = sum over rows of dy n
//
// All of it is bound by HBM: a row is read once, stays in registers (a lane
// holds up to eight 16-byte vectors) and is written once.  16,384 rows of 4096
// bf16: forward with residual, kept, 0.61 GB in 107 us (5.7 TB/s); restore 0.20 GB
// in 35; backward 0.47 GB in 95 (5.0 TB/s), its fold of 512 partial rows 5.  A wavefront takes a
// row where the row fits one, so that rows need no barrier; longer rows take 4
// or 8 wavefronts.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "launch.h"
#include "rows.h"

namespace zs {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kTinyMax = 0x1p-100f;
constexpr uint32_t kMaxDim = 1u << 14;

struct NormArgs {
  const void *x, *residual, *gain;
  void *h, *out;
  uint8_t* codes;
  float *scales, *rstd;
  uint64_t n_rows;
  uint32_t dim, blocks;  // blocks: scales of a row
  double eps;
};

struct BackwardArgs {
  const void *dy, *gain, *h, *upstream;
  const uint8_t* codes;
  const float *scales, *rstd;
  void* dx;
  float* partial;  // [gridDim.x][dim up to a multiple of 8]
  uint64_t n_rows;
  uint32_t dim, blocks;
};

typedef u32x2 __attribute__((aligned(1))) u32x2_any;
typedef uint32_t __attribute__((aligned(1))) u32_any;

// N codes of a row from element v N on.
template <int N, bool WHOLE>
__device__ __forceinline__ void store_codes(uint8_t* row, uint32_t v, uint32_t dim, const float (&x)[N]) {
  float y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) y[k] = k < N ? x[k % N] : 0.0f;
  const u32x2 c = encode8(y);
  const uint32_t e = v * N;
  if (e + N <= dim) {
    if constexpr (N == 8) *reinterpret_cast<u32x2_any*>(row + e) = c;
    else *reinterpret_cast<u32_any*>(row + e) = c[0];
  } else if (!WHOLE) {
#pragma unroll
    for (uint32_t k = 0; k < N; ++k)
      if (e + k < dim) row[e + k] = (uint8_t)(c[k >> 2] >> (8 * (k & 3)));
  }
}

template <int N, bool WHOLE>
__device__ __forceinline__ u32x2 load_codes(const uint8_t* row, uint32_t v, uint32_t dim) {
  const uint32_t e = v * N;
  u32x2 c = {0, 0};
  if (e + N <= dim) {
    if constexpr (N == 8) c = *reinterpret_cast<const u32x2_any*>(row + e);
    else c[0] = *reinterpret_cast<const u32_any*>(row + e);
  } else if (!WHOLE && e < dim) {
#pragma unroll
    for (uint32_t k = 0; k < N; ++k)
      if (e + k < dim) c[k >> 2] |= (uint32_t)row[e + k] << (8 * (k & 3));
  }
  return c;
}

// This thread's place: W wavefronts to a row, 4 rows to a block when W is 1.
template <int W>
struct Place {
  static constexpr int kThreads = W == 1 ? 256 : 64 * W, kRows = W == 1 ? 4 : 1;
  static __device__ __forceinline__ uint32_t lane() { return W == 1 ? threadIdx.x & 63 : threadIdx.x; }
  static __device__ __forceinline__ uint32_t row() { return W == 1 ? threadIdx.x >> 6 : 0; }
};

// VPT vectors to a lane: lane t of a row's 64 W holds vectors t, t + 64 W, ...
// WHOLE: rows are whole vectors.
template <int DT, int W, int VPT, bool WHOLE>
__global__ void __launch_bounds__(Place<W>::kThreads) norm_kernel(const NormArgs a) {
  constexpr int N = Lane<DT>::N;
  typedef typename Vec<DT>::T T;
  __shared__ double part[W];
  const uint32_t t = Place<W>::lane();
  for (uint64_t row = (uint64_t)blockIdx.x * Place<W>::kRows + Place<W>::row(); row < a.n_rows;
       row += (uint64_t)gridDim.x * Place<W>::kRows) {
    const uint64_t at = row * a.dim;
    u32x4 h[VPT], r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) h[i] = load_cut<DT, WHOLE>(static_cast<const T*>(a.x) + at, t + i * 64 * W, a.dim);
    if (a.residual) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) r[i] = load_cut<DT, WHOLE>(static_cast<const T*>(a.residual) + at, t + i * 64 * W, a.dim);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
#pragma unroll
        for (int k = 0; k < N; k += DT == ZERO_F32 ? 1 : 2) {
          const float s = Lane<DT>::get(h[i], k) + Lane<DT>::get(r[i], k);
          if constexpr (DT == ZERO_F32) h[i][k] = __float_as_uint(s);
          else h[i][k >> 1] = Vec<DT>::pack(s, Lane<DT>::get(h[i], k + 1) + Lane<DT>::get(r[i], k + 1));
        }
      }
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        // fp64: squares of the largest bf16 and fp32 values are beyond fp32
        const double v = (double)Lane<DT>::get(h[i], k);
        sum = fma(v, v, sum);
      }
    }
    sum = row_sum<W>(sum, part);
    const float rstd = (float)(1.0 / sqrt(sum / (double)a.dim + a.eps));
    if (a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const uint32_t v = t + i * 64 * W;
      float x[N], y[N];
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = Lane<DT>::get(h[i], k);
      if (a.h) store_cut<DT, false, WHOLE>(static_cast<T*>(a.h) + at, v, a.dim, x);
      const u32x4 g = load_cut<DT, WHOLE>(a.gain, v, a.dim);
#pragma unroll
      for (int k = 0; k < N; ++k) y[k] = x[k] * rstd * Lane<DT>::get(g, k);
      store_cut<DT, false, WHOLE>(static_cast<T*>(a.out) + at, v, a.dim, y);
      if (a.codes) {
        // magnitudes by their bits, where NaN is largest
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < N; ++k) top = max(top, __float_as_uint(x[k]) & 0x7FFFFFFFu);
        top = row16_max(top);  // 16 lanes hold 128 elements, of fp32 32 lanes
        if constexpr (N == 4) top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
        const float m = __uint_as_float(top);
        const bool live = !(m < kTinyMax);  // true for NaN
        const float inv = live ? kE4m3Max * (1.0f / m) : 0.0f;
        float c[N];
#pragma unroll
        for (int k = 0; k < N; ++k) c[k] = x[k] * inv;
        store_codes<N, WHOLE>(a.codes + at, v, a.dim, c);
        if (v % (128 / N) == 0 && v * N < a.dim)
          a.scales[row * a.blocks + v * N / 128] = live ? m * (1.0f / kE4m3Max) + (m - m) : 0.0f;  // not finite: NaN
      }
    }
  }
}

// y = n gain from the kept form.
template <int DT, int W, int VPT, bool WHOLE>
__global__ void __launch_bounds__(Place<W>::kThreads) restore_kernel(const NormArgs a) {
  constexpr int N = Lane<DT>::N;
  typedef typename Vec<DT>::T T;
  const uint32_t t = Place<W>::lane();
  for (uint64_t row = (uint64_t)blockIdx.x * Place<W>::kRows + Place<W>::row(); row < a.n_rows;
       row += (uint64_t)gridDim.x * Place<W>::kRows) {
    const uint64_t at = row * a.dim;
    const float rstd = a.rstd[row];
    u32x2 c[VPT];
    float s[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const uint32_t v = t + i * 64 * W;
      c[i] = load_codes<N, WHOLE>(a.codes + at, v, a.dim);
      s[i] = v * N < a.dim ? a.scales[row * a.blocks + v * N / 128] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const uint32_t v = t + i * 64 * W;
      float x[8], y[N];
      decode8(c[i], x);
      const u32x4 g = load_cut<DT, WHOLE>(a.gain, v, a.dim);
#pragma unroll
      for (int k = 0; k < N; ++k) y[k] = x[k] * s[i] * rstd * Lane<DT>::get(g, k);
      store_cut<DT, false, WHOLE>(static_cast<T*>(a.out) + at, v, a.dim, y);
    }
  }
}

// One row of the backward pass in registers.
template <int DT, int W, int VPT, bool KEPT, bool WHOLE>
struct Held {
  static constexpr int N = Lane<DT>::N;
  u32x4 d[VPT], up[VPT], h[KEPT ? 1 : VPT];
  u32x2 c[KEPT ? VPT : 1];
  float s[KEPT ? VPT : 1], rstd;

  __device__ __forceinline__ void load(const BackwardArgs& a, uint64_t row, uint32_t t) {
    typedef typename Vec<DT>::T T;
    const uint64_t at = row * a.dim;
    rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const uint32_t v = t + i * 64 * W;
      d[i] = load_cut<DT, WHOLE>(static_cast<const T*>(a.dy) + at, v, a.dim);
      if constexpr (KEPT) {
        c[i] = load_codes<N, WHOLE>(a.codes + at, v, a.dim);
        s[i] = v * N < a.dim ? a.scales[row * a.blocks + v * N / 128] : 0.0f;
      } else {
        h[i] = load_cut<DT, WHOLE>(static_cast<const T*>(a.h) + at, v, a.dim);
      }
    }
    if (a.upstream) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        up[i] = load_cut<DT, WHOLE>(static_cast<const T*>(a.upstream) + at, t + i * 64 * W, a.dim);
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) up[i] = u32x4{0, 0, 0, 0};
    }
  }
  __device__ __forceinline__ void normalised(int i, float (&n)[N]) const {
    if constexpr (KEPT) {
      float x[8];
      decode8(c[i], x);
#pragma unroll
      for (int k = 0; k < N; ++k) n[k] = x[k] * s[i] * rstd;
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) n[k] = Lane<DT>::get(h[i], k) * rstd;
    }
  }
};

// The backward pass's block: kRows rows at a time, of kLanes threads each.
template <int W, int VPT>
struct Group {
  static constexpr int kLanes = 64 * W, kRows = W == 1 ? 4 : W == 4 && VPT <= 2 ? 2 : 1, kThreads = kLanes * kRows;
};

// A block goes over groups of rows blockIdx, blockIdx + gridDim, ..., adds up
// dy n in registers and leaves one partial row for fold_kernel.  Held in fp32: dy n
// of a block's rows (some n_rows / 512 of them at most: fp64 would take twice the
// registers and the partial rows; of random numbers of one sign the result is within
// its own rounding up to a million rows) and dn n of a vector's 4 or 8 elements. The
// partial rows and the vectors are added in fp64.
template <int DT, int W, int VPT, bool KEPT, bool WHOLE>
__global__ void __launch_bounds__((Group<W, VPT>::kThreads)) backward_kernel(const BackwardArgs a) {
  constexpr int N = Lane<DT>::N, kLanes = Group<W, VPT>::kLanes, kRows = Group<W, VPT>::kRows;
  typedef typename Vec<DT>::T T;
  __shared__ double part[2][kRows][W];  // in turn, so that a row needs one barrier
  __shared__ float share[kRows > 1 ? (kRows - 1) * kLanes * N : 1];
  const uint32_t t = threadIdx.x % kLanes, g = threadIdx.x / kLanes;
  float dg[VPT][N] = {};
  // in registers, but for rows that fill them by themselves
  u32x4 held[VPT < 8 ? VPT : 1];
  const auto gain_at = [&](int i) { return load_cut<DT, WHOLE>(a.gain, t + i * kLanes, a.dim); };
  if constexpr (VPT < 8) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) held[i] = gain_at(i);
  }
  uint32_t turn = 0;
  for (uint64_t row0 = (uint64_t)blockIdx.x * kRows; row0 < a.n_rows; row0 += (uint64_t)gridDim.x * kRows, turn ^= 1) {
    const bool has = row0 + g < a.n_rows;
    const uint64_t row = has ? row0 + g : row0;  // behind the last row: one that is not counted
    Held<DT, W, VPT, KEPT, WHOLE> x;
    x.load(a, row, t);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const u32x4 gain = VPT < 8 ? held[i % (VPT < 8 ? VPT : 1)] : gain_at(i);
      float n[N], p = 0.0f;
      x.normalised(i, n);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float d = Lane<DT>::get(x.d[i], k), q = d * n[k];
        dg[i][k] += has ? q : 0.0f;
        p = fmaf(d * Lane<DT>::get(gain, k), n[k], p);  // dn as below: in few columns the two cancel
      }
      sum += (double)p;
    }
    const float mean = (float)(row_sum<W, false>(sum, part[turn][g]) / (double)a.dim);
    if (!has) continue;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const u32x4 gain = VPT < 8 ? held[i % (VPT < 8 ? VPT : 1)] : gain_at(i);
      float n[N], y[N];
      x.normalised(i, n);
#pragma unroll
      for (int k = 0; k < N; ++k)
        y[k] = fmaf(x.rstd, fmaf(-n[k], mean, Lane<DT>::get(x.d[i], k) * Lane<DT>::get(gain, k)), Lane<DT>::get(x.up[i], k));
      store_cut<DT, false, WHOLE>(static_cast<T*>(a.dx) + row * a.dim, t + i * kLanes, a.dim, y);
    }
  }
  // the block's rows together, a vector of each at a time
  const uint64_t at = (uint64_t)blockIdx.x * ((a.dim + 7) / 8 * 8);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const uint32_t v = t + i * kLanes;
    if constexpr (kRows > 1) {
      __syncthreads();
      if (g > 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) share[((g - 1) * N + k) * kLanes + t] = dg[i][k];
      }
      __syncthreads();
      if (g > 0) continue;
#pragma unroll
      for (int r = 0; r < kRows - 1; ++r)
#pragma unroll
        for (int k = 0; k < N; ++k) dg[i][k] += share[(r * N + k) * kLanes + t];
    }
    if (v * N < a.dim) {
#pragma unroll
      for (int k = 0; k < N; k += 4)
        *reinterpret_cast<f32x4*>(a.partial + at + v * N + k) = f32x4{dg[i][k], dg[i][k + 1], dg[i][k + 2], dg[i][k + 3]};
    }
  }
}

// dgain[d] = sum of the partial rows: a block takes 32 columns, each of its 32
// groups of lanes every 32nd row.
constexpr int kFoldColumns = 32, kFoldGroups = 32;
__device__ __forceinline__ void store_any(int dtype, void* p, uint64_t e, float x) {
  if (dtype == ZERO_F16) Vec<ZERO_F16>::store1(p, e, x);
  else if (dtype == ZERO_BF16) Vec<ZERO_BF16>::store1(p, e, x);
  else Vec<ZERO_F32>::store1(p, e, x);
}
__global__ void __launch_bounds__(kFoldColumns * kFoldGroups) fold_kernel(const float* partial, uint32_t n, uint32_t dim,
                                                                          void* dgain, int dtype) {
  __shared__ double s[kFoldGroups][kFoldColumns];
  const uint32_t c = threadIdx.x % kFoldColumns, g = threadIdx.x / kFoldColumns;
  const uint32_t d = blockIdx.x * kFoldColumns + c;
  const uint32_t row = (dim + 7) / 8 * 8;
  double sum = 0.0;
  if (d < dim) {
#pragma unroll 8
    for (uint32_t i = g; i < n; i += kFoldGroups) sum += (double)partial[(uint64_t)i * row + d];
  }
  s[g][c] = sum;
  __syncthreads();
  for (uint32_t half = kFoldGroups / 2; half > 0; half /= 2) {
    if (g < half) s[g][c] += s[g + half][c];
    __syncthreads();
  }
  if (g == 0 && d < dim) store_any(dtype, dgain, d, (float)s[0][c]);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
// Wavefronts to a row and vectors to a lane.  Measured over 64 M elements bf16, from 16
// bits the forward pass (with residual, kept) and the backward pass, and the next choice
// on either side:
//   dim 1024   1 x 2  111 and  77 us;  4 x 1  117 and 101
//   dim 2048   4 x 1  108 and  77;     1 x 4  112 and  78
//   dim 4096   4 x 2  107 and  77;     8 x 1  108 and  78;   1 x 8  125 and 112
//   dim 8192   4 x 4  111 and  81;     8 x 2  110 and  88
//   dim 16384  8 x 4  115 and  91;     4 x 8  123 and 118
// (8 x 1 at 4096 is 4% faster backward from the kept form, 90 us for 94, and 8% slower
// at restoring, 41 for 38.  Four rows take the same time either way.)
template <int DT, typename F>
void by_width(uint32_t dim, F fn) {
  const uint32_t vecs = (dim + Lane<DT>::N - 1) / Lane<DT>::N;
  const auto go = [&](auto w, auto v) {
    // (with eight vectors to a lane the kernels of whole vectors spill registers)
    if constexpr (decltype(v)::value < 8) {
      if (dim % Lane<DT>::N == 0) return fn(w, v, std::true_type{});
    }
    fn(w, v, std::false_type{});
  };
  if (vecs <= 64) go(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
  else if (vecs <= 128) go(std::integral_constant<int, 1>{}, std::integral_constant<int, 2>{});
  else if (vecs <= 256) go(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
  else if (vecs <= 512) go(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
  else if (vecs <= 1024) go(std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
  else if (vecs <= 2048) go(std::integral_constant<int, 8>{}, std::integral_constant<int, 4>{});
  else if constexpr (DT == ZERO_F32) go(std::integral_constant<int, 8>{}, std::integral_constant<int, 8>{});
}

int check_rows(uint64_t n_rows, uint32_t dim, int dtype, const char* who) {
  if (!known_dtype(dtype)) return fail(ZERO_EINVAL, "%s: unknown dtype %d", who, dtype);
  if (dim == 0 || dim > kMaxDim) return fail(ZERO_EINVAL, "%s: dim %u outside [1, %u]", who, dim, kMaxDim);
  if (n_rows > UINT64_MAX / 8 / dim) return fail(ZERO_EINVAL, "%s: n_rows * dim overflows", who);
  return ZERO_OK;
}

uint32_t scales_of(uint32_t dim) { return (dim + ZERO_QBLOCK - 1) / ZERO_QBLOCK; }

// Blocks of the backward pass.  Each leaves a partial row of dgain in fp32, so
// there are 512 at most.  256, 512, 768 and 1024 of them take, of 16,384 rows of 4096
// bf16, two rows at a time, from 16 bits 84, 78, 82 and 81 us and from the kept form
// with an upstream gradient 92, 94, 97 and 99; of 999 rows of 5003 fp16, a row at a
// time, 20, 17, 19 and 22.
constexpr uint64_t kBackwardBlocks = 512;

}  // namespace
}  // namespace zs

using namespace zs;

extern "C" int zero_rms_norm(const void* x, const void* residual, const void* gain, int dtype, uint64_t n_rows,
                             uint32_t dim, double eps, void* h, void* out, float* rstd, uint8_t* codes, float* scales,
                             hipStream_t stream) {
  static const char* who = "zero_rms_norm";
  clear_error();
  int rc = check_rows(n_rows, dim, dtype, who);
  if (rc) return rc;
  if (!std::isfinite(eps) || eps < 0.0) return fail(ZERO_EINVAL, "%s: eps must be finite and >= 0", who);
  if (n_rows == 0) return ZERO_OK;
  if (!x || !gain || !out) return fail(ZERO_EINVAL, "%s: x, gain and out must be given", who);
  if (!residual != !h) return fail(ZERO_EINVAL, "%s: residual and h go together", who);
  if (!codes != !scales) return fail(ZERO_EINVAL, "%s: codes and scales go together", who);
  const uint32_t b = dtype_bytes(dtype);
  if (!multiple_of(x, b) || !multiple_of(residual, b) || !multiple_of(gain, b) || !multiple_of(h, b) ||
      !multiple_of(out, b) || !multiple_of(rstd, 4) || !multiple_of(scales, 4))
    return fail(ZERO_EINVAL, "%s: an array is not aligned to its elements", who);
  if ((rc = begin_launch())) return rc;
  const NormArgs a = {x, residual, gain, h, out, codes, scales, rstd, n_rows, dim, scales_of(dim), eps};
  with_dtype(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    by_width<DT>(dim, [&](auto w, auto v, auto whole) {
      constexpr int W = decltype(w)::value, VPT = decltype(v)::value;
      constexpr bool WHOLE = decltype(whole)::value;
      const uint64_t blocks = (n_rows + Place<W>::kRows - 1) / Place<W>::kRows;
      hipLaunchKernelGGL((norm_kernel<DT, W, VPT, WHOLE>), chunk_grid(std::min<uint64_t>(blocks, 1u << 20), 0),
                         Place<W>::kThreads, 0, stream, a);
    });
  });
  return launch_status(who);
}

extern "C" int zero_rms_norm_restore(const uint8_t* codes, const float* scales, const float* rstd, const void* gain,
                                     int dtype, uint64_t n_rows, uint32_t dim, void* out, hipStream_t stream) {
  static const char* who = "zero_rms_norm_restore";
  clear_error();
  int rc = check_rows(n_rows, dim, dtype, who);
  if (rc) return rc;
  if (n_rows == 0) return ZERO_OK;
  if (!codes || !scales || !rstd || !gain || !out)
    return fail(ZERO_EINVAL, "%s: codes, scales, rstd, gain and out must be given", who);
  const uint32_t b = dtype_bytes(dtype);
  if (!multiple_of(gain, b) || !multiple_of(out, b) || !multiple_of(rstd, 4) || !multiple_of(scales, 4))
    return fail(ZERO_EINVAL, "%s: an array is not aligned to its elements", who);
  if ((rc = begin_launch())) return rc;
  NormArgs a = {};
  a.codes = const_cast<uint8_t*>(codes);
  a.scales = const_cast<float*>(scales);
  a.rstd = const_cast<float*>(rstd);
  a.gain = gain;
  a.out = out;
  a.n_rows = n_rows;
  a.dim = dim;
  a.blocks = scales_of(dim);
  with_dtype(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    by_width<DT>(dim, [&](auto w, auto v, auto whole) {
      constexpr int W = decltype(w)::value, VPT = decltype(v)::value;
      constexpr bool WHOLE = decltype(whole)::value;
      const uint64_t blocks = (n_rows + Place<W>::kRows - 1) / Place<W>::kRows;
      hipLaunchKernelGGL((restore_kernel<DT, W, VPT, WHOLE>), chunk_grid(std::min<uint64_t>(blocks, 1u << 20), 0),
                         Place<W>::kThreads, 0, stream, a);
    });
  });
  return launch_status(who);
}

extern "C" int zero_rms_norm_workspace_bytes(uint64_t n_rows, uint32_t dim, uint64_t* bytes) {
  clear_error();
  if (!bytes) return fail(ZERO_EINVAL, "zero_rms_norm_workspace_bytes: bytes is NULL");
  if (dim == 0 || dim > kMaxDim)
    return fail(ZERO_EINVAL, "zero_rms_norm_workspace_bytes: dim %u outside [1, %u]", dim, kMaxDim);
  *bytes = std::max<uint64_t>(std::min(n_rows, kBackwardBlocks), 1) * ((dim + 7) / 8 * 8) * 4;
  return ZERO_OK;
}

extern "C" int zero_rms_norm_backward(const zero_rms_norm_backward_args* p, hipStream_t stream) {
  static const char* who = "zero_rms_norm_backward";
  clear_error();
  if (!p) return fail(ZERO_EINVAL, "%s: args is NULL", who);
  int rc = check_rows(p->n_rows, p->dim, p->dtype, who);
  if (rc) return rc;
  if (!p->dgain) return fail(ZERO_EINVAL, "%s: dgain must be given", who);
  const uint32_t b = dtype_bytes(p->dtype);
  if (!multiple_of(p->dgain, b)) return fail(ZERO_EINVAL, "%s: dgain is not aligned to its elements", who);
  const uint64_t blocks = std::min(p->n_rows, kBackwardBlocks);
  if (p->n_rows > 0) {
    if (!p->dy || !p->gain || !p->rstd || !p->dx) return fail(ZERO_EINVAL, "%s: dy, gain, rstd and dx must be given", who);
    if (!p->codes != !p->scales) return fail(ZERO_EINVAL, "%s: codes and scales go together", who);
    if (!p->h == !p->codes) return fail(ZERO_EINVAL, "%s: either h or codes must be given", who);
    if (!multiple_of(p->dy, b) || !multiple_of(p->gain, b) || !multiple_of(p->h, b) || !multiple_of(p->upstream, b) ||
        !multiple_of(p->dx, b) || !multiple_of(p->rstd, 4) || !multiple_of(p->scales, 4))
      return fail(ZERO_EINVAL, "%s: an array is not aligned to its elements", who);
    const uint64_t need = blocks * ((p->dim + 7) / 8 * 8) * 4;
    if (!p->workspace) return fail(ZERO_EINVAL, "%s: workspace is NULL", who);
    if (p->workspace_bytes < need)
      return fail(ZERO_EINVAL, "%s: workspace needs %llu bytes, got %zu", who, (unsigned long long)need, p->workspace_bytes);
    if (!multiple_of(p->workspace, 256)) return fail(ZERO_EINVAL, "%s: workspace must be 256-byte aligned", who);
  }
  if ((rc = begin_launch())) return rc;
  uint32_t parts = 0;
  if (p->n_rows > 0) {
    const BackwardArgs a = {p->dy, p->gain, p->h, p->upstream, p->codes, p->scales, p->rstd, p->dx,
                            static_cast<float*>(p->workspace), p->n_rows, p->dim, scales_of(p->dim)};
    with_dtype(p->dtype, [&](auto dt) {
      constexpr int DT = decltype(dt)::value;
      by_width<DT>(p->dim, [&](auto w, auto v, auto whole) {
        constexpr int W = decltype(w)::value, VPT = decltype(v)::value;
        constexpr bool WHOLE = decltype(whole)::value;
        typedef Group<W, VPT> G;
        parts = (uint32_t)std::min<uint64_t>((p->n_rows + G::kRows - 1) / G::kRows, kBackwardBlocks);
        if (p->codes)
          hipLaunchKernelGGL((backward_kernel<DT, W, VPT, true, WHOLE>), parts, G::kThreads, 0, stream, a);
        else
          hipLaunchKernelGGL((backward_kernel<DT, W, VPT, false, WHOLE>), parts, G::kThreads, 0, stream, a);
      });
    });
    if ((rc = launch_status(who))) return rc;
  }
  hipLaunchKernelGGL(fold_kernel, (p->dim + kFoldColumns - 1) / kFoldColumns, kFoldColumns * kFoldGroups, 0,
                     stream,
                     static_cast<const float*>(p->workspace), parts, p->dim, p->dgain, p->dtype);
  return launch_status(who);
}
