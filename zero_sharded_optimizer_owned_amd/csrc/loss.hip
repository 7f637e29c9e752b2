// Losses on token log-probabilities and their gradient of the logits.
//
// For a row x of logits, its target t, a temperature T and any reference z,
//   S = sum_j exp((x_j - z) / T),  lp = (x_t - z) / T - ln S,
//   d lp / d x_j = ([j = t] - exp((x_j - z) / T) / S) / T,
// so a loss that is a function of the rows' lp has the gradient
//   dx_j = coef * ([j = t] - p_j)
// with one number `coef` per row.  Everything over the vocabulary is one sum
// and one product per element; what makes the losses differ is a few dozen
// operations per row, done in fp64 by one thread, since the lp of hundreds of
// tokens are added and their differences exponentiated.
//
// The reference is the target's own logit: it needs no pass over the row, is
// the same for every thread (partial sums simply add), and lp = -ln S.  It
// serves unless the row's maximum is some 40 T above it; a sum that is not
// below 2^60 (NaN, infinity) sends the row through a second form whose
// reference is the maximum, found as it goes (8192 rows of 32,000 bf16 that all
// need it: log-probabilities 197 us instead of 77).
//
// The elements are fp32, exp is the hardware's 2^x with log2(e) / T as its
// factor.  The difference to the reference comes first, so that errors go with
// it and not with the logits' size: the target's own term is exactly 1, lp is
// never above 0 and a shift of all logits changes nothing.  (x c - x_t c with
// the second product rounded to fp32 costs 2^-24 |x_t| / T of lp, and the whole
// row where that product overflows.)  In the sums the factor has a second word:
// fp32's error of log2(e), 1.3e-8, moves every row's ln S the same way
// (measured on 500-token sequences: rewards 5e-6 off without it, 4e-7 with
// it).  Every call forms a row's sum alike: the reference model's
// log-probabilities and the policy's agree to the bit where the logits do.
// A thread adds a vector's 4 or 8 elements in fp32, and the vectors that it
// holds in registers (at most 16); everything past that is added up in fp64.
//
// A row whose target is outside [0, vocab), or whose logits are all -inf,
// counts for nothing: lp 0, gradient 0, and nothing of it is looked at.  NaN
// and +inf logits in a row that counts give NaN.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <limits>
#include <type_traits>

#include "internal.h"
#include "launch.h"
#include "vec.h"

namespace zs {
namespace {

constexpr double kLog2e = 1.4426950408889634;

struct Logits {
  const void* x;
  uint64_t n_rows, stride;  // stride in elements
  uint32_t vocab;
  const int64_t* targets;
  float c;           // log2(e) / T
  float c_hi, c_lo;  // the same in two words: the fp32 value below it and the rest, which is
                     // held above 0, so that d = -inf gives -inf in both
  double inv_t;  // 1 / T
};

// One row of `vocab` elements: n_vec 16-byte vectors from the first 128-byte
// boundary on, and up to 70 elements before and after them, one to a thread.
// Rows of most vocabularies start anywhere.  Vectors from the row's own start
// run 25-30% slower there (4096 rows of 50,001 bf16: policy loss 210 us, so 168;
// 2048 rows of 128,001: 246 us and, preference loss, 362; so 198 and 276, as for
// 128,000).
constexpr uint32_t kRowAlign = 128;

template <int DT>
struct Row {
  const void* x;       // the row's first element
  const void* v;       // the first vector
  uint32_t head;       // elements before it
  uint32_t n_vec, vocab;
  static constexpr uint32_t N = Lane<DT>::N;

  __device__ __forceinline__ Row(const Logits& a, uint64_t row) {
    typedef typename Vec<DT>::T T;
    const T* p = static_cast<const T*>(a.x) + row * a.stride;
    vocab = a.vocab;
    head = min((uint32_t)(-reinterpret_cast<uintptr_t>(p) & (kRowAlign - 1u)) / (uint32_t)sizeof(T), vocab);
    x = p;
    v = p + head;
    n_vec = (vocab - head) / N;
  }
  // Thread t's element beside the vectors, if it has one.
  __device__ __forceinline__ bool has_side(uint32_t t) const { return t < vocab - N * n_vec; }
  __device__ __forceinline__ uint32_t side(uint32_t t) const { return t < head ? t : N * n_vec + t; }
};

// ln s for finite s > 0 (NaN for NaN), and e^x - 1 and e^x, in fp64 to about
// 1e-14, relative: s = 2^e m with m next to 1 and ln m = 2 artanh((m - 1) /
// (m + 1)) by its series; x = n ln 2 + r and e^r - 1 by its Taylor polynomial.
// They take some 20 registers where the general functions take 100, which a
// block that holds a row in registers does not have.
__device__ __forceinline__ double ln(double s) {
  int e = __builtin_amdgcn_frexp_exp(s);
  double m = __builtin_amdgcn_frexp_mant(s);
  if (m < 0.70710678118654752) {
    m += m;
    --e;
  }
  const double t = (m - 1.0) / (m + 1.0), q = t * t;
  double p = 1.0 / 17;
  p = fma(p, q, 1.0 / 15);
  p = fma(p, q, 1.0 / 13);
  p = fma(p, q, 1.0 / 11);
  p = fma(p, q, 1.0 / 9);
  p = fma(p, q, 1.0 / 7);
  p = fma(p, q, 1.0 / 5);
  p = fma(p, q, 1.0 / 3);
  const double u = t + t;
  return fma((double)e, 0.693147180559945309, fma(u * q, p, u));
}

struct Exp {
  double value, minus1;
};

__device__ __forceinline__ Exp exp_both(double x) {
  x = x < -800.0 ? -800.0 : x > 800.0 ? 800.0 : x;  // beyond both ends of fp64; NaN stays
  const double n = rint(x * 1.44269504088896341);
  // ln 2 as its fp32 value, whose product with n is exact, and the rest
  const double r = fma(n, 1.90465429995776805e-9, fma(n, -0.693147182464599609375, x));
  double p = 1.0 / 479001600;
  p = fma(p, r, 1.0 / 39916800);
  p = fma(p, r, 1.0 / 3628800);
  p = fma(p, r, 1.0 / 362880);
  p = fma(p, r, 1.0 / 40320);
  p = fma(p, r, 1.0 / 5040);
  p = fma(p, r, 1.0 / 720);
  p = fma(p, r, 1.0 / 120);
  p = fma(p, r, 1.0 / 24);
  p = fma(p, r, 1.0 / 6);
  p = fma(p, r, 0.5);
  p = fma(p * r, r, r);  // e^r - 1
  const double value = ldexp(1.0 + p, (int)n);
  return {value, n == 0.0 ? p : value - 1.0};
}

// A value that is the same in every thread, in a scalar register: rows in
// registers leave none to spare.
__device__ __forceinline__ float uniform(float x) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

// A running (maximum, sum of exp2((x - max) c)).
struct MaxSum {
  float m;
  double s;
};

__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.0f : m; }

// exp((x - z) / T) of the sum.
__device__ __forceinline__ float term(float x, float z, const Logits& in) {
  const float d = x - z;
  return __builtin_amdgcn_exp2f(fmaf(d, in.c_hi, d * in.c_lo));
}

__device__ __forceinline__ MaxSum join(const MaxSum& a, const MaxSum& b, const Logits& in) {
  const float m = fmaxf(a.m, b.m), z = finite_or_zero(m);
  return {m, a.s * (double)term(a.m, z, in) + b.s * (double)term(b.m, z, in)};
}

// Over a block of W wavefronts, in a fixed tree; the result is in every thread.
template <int W>
__device__ __forceinline__ MaxSum block_join(MaxSum v, const Logits& in) {
  __shared__ MaxSum part[W];
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = join(v, MaxSum{__shfl_xor(v.m, off, 64), __shfl_xor(v.s, off, 64)}, in);
  __syncthreads();  // `part` may still be read for the row before
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int i = 1; i < W; ++i) v = join(v, part[i], in);
  return v;
}

// coef at the target's place, `at` elements after the first of these (if it is
// one of them).
template <int N>
__device__ __forceinline__ void add_at_target(float (&dx)[N], uint32_t at, float coef) {
  if (at < N) {
#pragma unroll
    for (int i = 0; i < N; ++i) dx[i] += at == (uint32_t)i ? coef : 0.0f;
  }
}

// Sum of one double per thread over a block of W wavefronts, in a fixed tree;
// in every thread.
template <int W = kWavesPerBlock>
__device__ __forceinline__ double block_sum(double x) {
  __shared__ double part[W];
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x = x + __shfl_xor(x, off, 64);
  if (W == 1) return x;
  __syncthreads();  // `part` may still be read for the sum before
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  x = part[0];
#pragma unroll
  for (int i = 1; i < W; ++i) x = x + part[i];
  return x;
}

// The sum with reference z over a row by a block of 64 W threads, in every
// thread.
template <int DT, int W = kWavesPerBlock>
__device__ __forceinline__ double row_sum(const Row<DT>& r, float z, const Logits& in) {
  const uint32_t t = threadIdx.x;
  double s = 0.0;
#pragma unroll 4
  for (uint32_t v = t; v < r.n_vec; v += 64 * W) {
    const auto raw = load16_any(r.v, v);
    float e = 0.0f;
#pragma unroll
    for (int k = 0; k < Lane<DT>::N; ++k) e += term(Lane<DT>::get(raw, k), z, in);
    s += (double)e;
  }
  if (r.has_side(t)) s += (double)term(Vec<DT>::load1(r.x, r.side(t)), z, in);
  return block_sum<W>(s);
}

// (reference, sum) with the row's maximum as the reference, found on the way;
// (0, 0) when every logit is -inf.
template <int DT, int W = kWavesPerBlock>
__device__ __forceinline__ MaxSum row_max_sum(const Row<DT>& r, const Logits& in) {
  constexpr int N = Lane<DT>::N;
  const uint32_t t = threadIdx.x;
  MaxSum own = {-INFINITY, 0.0};
  // the sum so far goes over to the larger maximum, then a vector's terms join it
  auto raise = [&](float top) {
    const float nm = fmaxf(own.m, top), z = finite_or_zero(nm);
    own.s *= (double)term(own.m, z, in);
    own.m = nm;
    return z;
  };
  for (uint32_t v = t; v < r.n_vec; v += 64 * W) {
    const auto raw = load16_any(r.v, v);
    float top = -INFINITY, e = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) top = fmaxf(top, Lane<DT>::get(raw, k));
    const float z = raise(top);
#pragma unroll
    for (int k = 0; k < N; ++k) e += term(Lane<DT>::get(raw, k), z, in);
    own.s += (double)e;
  }
  if (r.has_side(t)) {
    const float x = Vec<DT>::load1(r.x, r.side(t)), z = raise(x);
    own.s += (double)term(x, z, in);
  }
  MaxSum all = block_join<W>(own, in);
  all.m = finite_or_zero(all.m);
  return all;
}

// A sum that the reference xt serves (false for NaN).
__device__ __forceinline__ bool served(double s) { return s < 0x1p60; }

// A row's reference and sum; lp and whether the row counts follow.
struct RowSum {
  float z;
  double s;
  __device__ __forceinline__ bool counts() const { return s != 0.0; }  // true for NaN
  __device__ __forceinline__ double logp(float xt, const Logits& in) const {
    return counts() ? ((double)xt - (double)z) * in.inv_t - ln(s) : 0.0;
  }
};

// Where the target's logit has been tried and does not serve.
template <int DT, int W = kWavesPerBlock>
__device__ __forceinline__ RowSum row_by_max(const Row<DT>& r, const Logits& in) {
  const MaxSum ms = row_max_sum<DT, W>(r, in);
  return {ms.m, ms.s};
}

template <int DT, int W = kWavesPerBlock>
__device__ __forceinline__ RowSum row_reduce(const Row<DT>& r, float xt, const Logits& in) {
  const double s = row_sum<DT, W>(r, xt, in);
  return served(s) ? RowSum{xt, s} : row_by_max<DT, W>(r, in);
}

// dx = coef ([j = t] - p) over the row by the block; zeros when coef is 0.
// `out` may be the row itself: each element is read and written by one thread.
template <int DT, int W, bool NT>
__device__ __forceinline__ void row_gradient(const Row<DT>& r, void* out, int64_t target, const RowSum& rs, float c,
                                             float coef) {
  const uint32_t t = threadIdx.x;
  const float k = (float)(-(double)coef / rs.s);
  void* out_v = static_cast<typename Vec<DT>::T*>(out) + r.head;
  for (uint32_t v = t; v < r.n_vec; v += 64 * W) {
    float dx[Lane<DT>::N] = {};
    if (coef != 0.0f) {
      const auto raw = load16_any<NT>(r.v, v);
#pragma unroll
      for (int i = 0; i < Lane<DT>::N; ++i) dx[i] = k * __builtin_amdgcn_exp2f((Lane<DT>::get(raw, i) - rs.z) * c);
      add_at_target(dx, (uint32_t)target - r.head - r.N * v, coef);
    }
    store16_any<DT, NT>(out_v, v, dx);
  }
  if (r.has_side(t)) {
    const uint32_t j = r.side(t);
    float dx = 0.0f;
    if (coef != 0.0f) {
      dx = k * __builtin_amdgcn_exp2f((Vec<DT>::load1(r.x, j) - rs.z) * c);
      if (j == target) dx += coef;
    }
    Vec<DT>::store1(out, j, dx);
  }
}

// A row spread over a block of 64 W threads, K vectors and at most one element
// beside them per thread.  Threads past the row's last vector load that one
// again and count it as 0, so that all loads are issued before the first is
// waited for, without branches; steps of the upper half that no thread of the
// block needs are left out.
// NT: loaded with the nontemporal hint, where no later pass reads them again
// (log-probabilities of 4096 x 128,000: 162 us without it, 155 with it).
template <int DT, int W, int K, bool NT>
struct Spread {
  static constexpr uint32_t kStep = 64 * W;
  // The largest block takes rows beyond its registers too: what is past them
  // is read where it is needed.
  static constexpr bool kRest = W == 16 && K == 16;
  u32x4 x[K];
  float side;

  static __device__ __forceinline__ bool step(int k, const Row<DT>& r) { return k < K / 2 || k * kStep < r.n_vec; }

  __device__ __forceinline__ Spread(const Row<DT>& r, uint32_t t) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (step(k, r)) x[k] = load16_any<NT>(r.v, min(k * kStep + t, r.n_vec - 1));
    side = r.has_side(t) ? Vec<DT>::load1(r.x, r.side(t)) : 0.0f;
  }

  // This thread's share of the sum; term(x) is an element's, and keep(k, i, q)
  // sees it (k = K: the one beside the vectors).
  template <typename T, typename F>
  __device__ __forceinline__ double sum(const Row<DT>& r, uint32_t t, T term, F keep) const {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (step(k, r)) {
        float part = 0.0f;
#pragma unroll
        for (int i = 0; i < Lane<DT>::N; ++i) {
          const float q = term(Lane<DT>::get(x[k], i));
          keep(k, i, q);
          part += q;
        }
        s += k * kStep + t < r.n_vec ? part : 0.0f;
      }
    }
    const float q = term(side);
    keep(K, 0, q);
    double all = (double)(r.has_side(t) ? s + q : s);
    if constexpr (kRest) {
#pragma unroll 2
      for (uint32_t v = K * kStep + t; v < r.n_vec; v += kStep) {
        const auto y = load16_any(r.v, v);
        float part = 0.0f;
#pragma unroll
        for (int i = 0; i < Lane<DT>::N; ++i) part += term(Lane<DT>::get(y, i));
        all += (double)part;
      }
    }
    return all;
  }
};

// Calls fn with the block (wavefronts, vectors per thread) whose threads hold a
// row in registers: 64 elements each, 128 of 16-bit rows past 65,536 elements,
// 16 up to 2048 elements, where twice as many blocks to a CU hide the rows'
// fp64 arithmetic (8192 rows of 1000 bf16: policy loss 25.3 us, so 17.8).
// False if the row is so short that no vector is sure to be left.
template <int DT, typename F>
bool with_spread(uint32_t vocab, F fn) {
  using std::integral_constant;
  using K = integral_constant<int, 64 / Lane<DT>::N>;
  if (vocab < 128) return false;
  if (vocab <= 64 * 2 * 16) fn(integral_constant<int, 2>{}, integral_constant<int, 16 / Lane<DT>::N>{});
  else if (vocab <= 64 * 2 * 64) fn(integral_constant<int, 2>{}, K{});
  else if (vocab <= 64 * 4 * 64) fn(integral_constant<int, 4>{}, K{});
  else if (vocab <= 64 * 8 * 64) fn(integral_constant<int, 8>{}, K{});
  else if (vocab <= 64 * 16 * 64) fn(integral_constant<int, 16>{}, K{});
  else fn(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  return true;
}

// One block per row, as many rows to a launch as its threads may number; each
// XCD takes one contiguous run of them (against rows dealt in turn: policy
// loss of 8192 x 128,000 715 to 708 us, preference loss of 8067 x 32,000 234
// to 226; its second pass is 1% slower so, and deals).
constexpr uint64_t kMostRows = 1u << 21;

__device__ __forceinline__ bool in_vocab(int64_t target, uint32_t vocab) { return target >= 0 && target < (int64_t)vocab; }

// ---------------------------------------------------------------------------
// Log-probabilities of the targets.
// ---------------------------------------------------------------------------
// What the preference loss keeps of a row between its passes.
struct RowStats {
  double lp, sum;
  float z, coef;
};

struct LogpArgs {
  Logits in;
  uint64_t row0;  // of a launch's first block
  float* logp;
  RowStats* stats;  // NULL unless a later pass needs them
};

__device__ __forceinline__ void logp_finish(const LogpArgs& a, uint64_t row, const RowSum& rs, float xt) {
  const double lp = rs.logp(xt, a.in);
  a.logp[row] = (float)lp;
  if (a.stats) a.stats[row] = RowStats{lp, rs.s, rs.z, 0.0f};  // sum 0: does not count
}

template <int DT>
__global__ void __launch_bounds__(kBlock) logp_kernel(const LogpArgs a) {
  for (uint64_t row = blockIdx.x; row < a.in.n_rows; row += gridDim.x) {
    const int64_t target = a.in.targets[row];
    RowSum rs = {0.0f, 0.0};
    float xt = 0.0f;
    if (in_vocab(target, a.in.vocab)) {  // the same for the whole block
      const Row<DT> r(a.in, row);
      xt = Vec<DT>::load1(r.x, (uint64_t)target);
      rs = row_reduce(r, xt, a.in);
    }
    if (threadIdx.x == 0) logp_finish(a, row, rs, xt);
  }
}

// NT: nothing reads the logits again.
template <int DT, int W, int K, bool NT>
__global__ void __launch_bounds__(64 * W, K * Lane<DT>::N <= 16 ? 8 : 4) logp_spread_kernel(const LogpArgs a) {
  const uint32_t t = threadIdx.x;
  const uint64_t row = a.row0 + xcd_contiguous(blockIdx.x, gridDim.x);
  const int64_t target = a.in.targets[row];
  RowSum rs = {0.0f, 0.0};
  float xt = 0.0f;
  if (in_vocab(target, a.in.vocab)) {
    const Row<DT> r(a.in, row);
    xt = Vec<DT>::load1(r.x, (uint64_t)target);
    const Spread<DT, W, K, NT> x(r, t);
    rs = {xt, block_sum<W>(x.sum(r, t, [&](float v) { return term(v, xt, a.in); }, [](int, int, float) {}))};
    if (!__builtin_amdgcn_readfirstlane(served(rs.s))) rs = row_by_max<DT, W>(r, a.in);
  }
  if (t == 0) logp_finish(a, row, rs, xt);
}

template <int DT, bool NT>
void launch_logp(LogpArgs a, hipStream_t s) {
  const bool done = with_spread<DT>(a.in.vocab, [&](auto w, auto k) {
    constexpr int W = decltype(w)::value, K = decltype(k)::value;
    for (a.row0 = 0; a.row0 < a.in.n_rows; a.row0 += kMostRows)
      hipLaunchKernelGGL((logp_spread_kernel<DT, W, K, NT>), (uint32_t)std::min(kMostRows, a.in.n_rows - a.row0),
                         64 * W, 0, s, a);
  });
  if (!done) hipLaunchKernelGGL(logp_kernel<DT>, chunk_grid(a.in.n_rows, 0), kBlock, 0, s, a);
}

// ---------------------------------------------------------------------------
// Clipped policy loss with a KL term: the forward and the gradient of a row
// by one block.
// ---------------------------------------------------------------------------
struct PolicyTerms {
  double gain, kl, clipped;  // each times weight / divisor
};

struct PolicyArgs {
  Logits in;
  uint64_t row0;  // of a launch's first block
  const float *old_logp, *ref_logp, *advantage, *weight;
  double inv_divisor, low, high, kl_coef, grad_scale;
  float *logp, *stats;
  void* dlogits;
  uint64_t dstride;
  PolicyTerms* terms;
  uint64_t* ticket;  // NULL: a launch of its own adds up the terms
};

// What a row brings besides its logits, loaded ahead of them: each would be a
// round trip to memory of its own where it is used.
struct PolicyRow {
  float weight, advantage, old_logp, ref_logp;
};

__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs& a, uint64_t row) {
  return {a.weight ? a.weight[row] : 1.0f, a.advantage[row], a.old_logp[row], a.ref_logp ? a.ref_logp[row] : 0.0f};
}

// The row's terms of the loss and its coefficient.
__device__ __forceinline__ float policy_terms(const PolicyArgs& a, const PolicyRow& in, double lp, PolicyTerms* out) {
  const double w = (double)in.weight * a.inv_divisor;
  if (w == 0.0) return 0.0f;
  const double adv = (double)in.advantage;
  double slope = 0.0;
  if (adv != 0.0) {  // 0 times an overflowed ratio is 0
    const double ratio = exp_both(lp - (double)in.old_logp).value;
    const double free = adv * ratio, held = adv * fmin(fmax(ratio, a.low), a.high);
    const bool clipped = held < free;
    out->gain = w * (clipped ? held : free);
    out->clipped = clipped ? w : 0.0;
    slope = clipped ? 0.0 : -free;
  }
  if (a.ref_logp) {
    const double d = (double)in.ref_logp - lp, e = exp_both(d).minus1;
    out->kl = w * (isinf(e) ? e : e - d);  // d is infinite too when lp is -inf
    if (a.kl_coef != 0.0) slope -= a.kl_coef * e;
  }
  return (float)(w * slope * a.grad_scale * a.in.inv_t);
}

// Stores and loads that are coherent across the chip: what one block of a launch
// leaves for another.
template <typename T>
__device__ __forceinline__ void put_agent(T* p, T x) {
  __hip_atomic_store(p, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ T get_agent(const T* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The row's log-probability and terms to memory, by one thread; its coefficient.
__device__ __forceinline__ float policy_finish(const PolicyArgs& a, uint64_t row, const PolicyRow& in, const RowSum& rs,
                                               float xt) {
  const double lp = rs.logp(xt, a.in);
  PolicyTerms terms = {0.0, 0.0, 0.0};
  const float coef = rs.counts() ? policy_terms(a, in, lp, &terms) : 0.0f;
  a.logp[row] = (float)lp;
  put_agent(&a.terms[row].gain, terms.gain);  // for the block that adds the terms up
  put_agent(&a.terms[row].kl, terms.kl);
  put_agent(&a.terms[row].clipped, terms.clipped);
  return coef;
}

template <int DT>
__device__ __forceinline__ typename Vec<DT>::T* policy_out(const PolicyArgs& a, uint64_t row) {
  return static_cast<typename Vec<DT>::T*>(a.dlogits) + row * a.dstride;
}

// The loss from all rows' terms, by one block of 64 W threads, each row's in a
// fixed place of a fixed tree.  COHERENT: the loads are coherent across the
// chip, where the last block of a launch adds up what others have just written.
template <int W, bool COHERENT>
__device__ __forceinline__ void policy_fold(const PolicyTerms* terms, uint64_t n, double kl_coef, float* stats) {
  __shared__ PolicyTerms part[W];
  auto get = [](const double* p) {
    if constexpr (COHERENT) return get_agent(p);
    else return *p;
  };
  PolicyTerms s = {0.0, 0.0, 0.0};
  auto add = [&](const PolicyTerms& x) {
    s.gain += x.gain;
    s.kl += x.kl;
    s.clipped += x.clipped;
  };
#pragma unroll 8
  for (uint64_t i = threadIdx.x; i < n; i += 64 * W)
    add({get(&terms[i].gain), get(&terms[i].kl), get(&terms[i].clipped)});
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1)
    add({__shfl_xor(s.gain, off, 64), __shfl_xor(s.kl, off, 64), __shfl_xor(s.clipped, off, 64)});
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < W; ++i) add(part[i]);
    put_agent(stats, (float)((kl_coef != 0.0 ? kl_coef * s.kl : 0.0) - s.gain));
    put_agent(stats + 1, (float)-s.gain);
    put_agent(stats + 2, (float)s.kl);
    put_agent(stats + 3, (float)s.clipped);
  }
}

constexpr int kFoldWaves = 16;
__global__ void __launch_bounds__(64 * kFoldWaves) policy_fold_kernel(const PolicyTerms* terms, uint64_t n,
                                                                      double kl_coef, float* stats) {
  policy_fold<kFoldWaves, false>(terms, n, kl_coef, stats);
}

// After a block's row is in memory (by thread 0): whether it was the last of
// the launch's rows.  The last one puts the count back to 0 for the next call.
// A count that did not start at 0 (a workspace that was never zeroed, or that
// two calls share at once) must not leave the stats of an earlier call: the
// first row's block sets them to NaN ahead of its own count, and so does every
// block that finds a count beyond the rows.  The count goes in steps of an odd
// constant, so that memory with small numbers in it is such a count too.
constexpr uint64_t kTicketStep = 0x9E3779B97F4A7C15u;
constexpr uint64_t odd_inverse(uint64_t x) {  // modulo 2^64, by Newton's iteration
  uint64_t y = x;
  for (int i = 0; i < 5; ++i) y *= 2 - x * y;
  return y;
}
static_assert(odd_inverse(kTicketStep) * kTicketStep == 1, "");

__device__ __forceinline__ void policy_spoil(const PolicyArgs& a) {
#pragma unroll
  for (int i = 0; i < 4; ++i) put_agent(a.stats + i, __builtin_nanf(""));
}

__device__ __forceinline__ bool policy_last(const PolicyArgs& a, uint64_t row) {
  if (!a.ticket) return false;
  if (row == 0) policy_spoil(a);
  const uint64_t before =
      __hip_atomic_fetch_add(a.ticket, kTicketStep, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) * odd_inverse(kTicketStep);
  if (before >= a.in.n_rows) policy_spoil(a);
  if (before + 1 != a.in.n_rows) return false;
  put_agent(a.ticket, (uint64_t)0);
  return true;
}

struct PolicyShared {
  float coef, scale;
  int last;
};

// What follows a row's sum, by a block of 64 W threads; the gradient reads the
// row again (mostly from the caches).
template <int DT, int W, bool NT>
__device__ __forceinline__ void policy_stream(const PolicyArgs& a, uint64_t row, const Row<DT>& r, int64_t target,
                                              const PolicyRow& in, float xt, const RowSum& rs, PolicyShared& sh) {
  __syncthreads();  // sh may still be read for the row before
  if (threadIdx.x == 0) {
    sh.coef = policy_finish(a, row, in, rs, xt);
    sh.last = policy_last(a, row);
  }
  __syncthreads();
  if (a.dlogits) row_gradient<DT, W, NT>(r, policy_out<DT>(a, row), target, rs, a.in.c, sh.coef);
}

template <int DT, bool NT>
__global__ void __launch_bounds__(kBlock) policy_kernel(const PolicyArgs a) {
  __shared__ PolicyShared sh;
  for (uint64_t row = blockIdx.x; row < a.in.n_rows; row += gridDim.x) {
    const int64_t target = a.in.targets[row];
    const bool in_range = in_vocab(target, a.in.vocab);
    const Row<DT> r(a.in, row);
    const PolicyRow in = policy_row(a, row);
    const float xt = in_range ? Vec<DT>::load1(r.x, (uint64_t)target) : 0.0f;
    const RowSum rs = in_range ? row_reduce(r, xt, a.in) : RowSum{0.0f, 0.0};
    policy_stream<DT, kWavesPerBlock, NT>(a, row, r, target, in, xt, rs, sh);
    if (sh.last) policy_fold<kWavesPerBlock, true>(a.terms, a.in.n_rows, a.kl_coef, a.stats);
  }
}

// A row held in registers, so that the logits are read once.  RAW keeps 16-bit
// logits, two to a register, and takes every exponential twice; otherwise the
// exponentials themselves stay.
template <int DT, int W, int K, bool RAW, bool NT>
__device__ __forceinline__ void policy_spread(const PolicyArgs& a, PolicyShared& sh) {
  const uint32_t t = threadIdx.x;
  const uint64_t row = a.row0 + xcd_contiguous(blockIdx.x, gridDim.x);
  const int64_t target = a.in.targets[row];
  const Row<DT> r(a.in, row);
  PolicyRow in = policy_row(a, row);
  if (!in_vocab(target, a.in.vocab))
    return policy_stream<DT, W, NT>(a, row, r, target, in, 0.0f, RowSum{0.0f, 0.0}, sh);
  float xt = Vec<DT>::load1(r.x, (uint64_t)target);
  Spread<DT, W, K, true> x(r, t);
  in = PolicyRow{uniform(in.weight), uniform(in.advantage), uniform(in.old_logp), uniform(in.ref_logp)};
  xt = uniform(xt);
  float e[RAW ? 1 : K][Lane<DT>::N], side = 0.0f;
  const double s = x.sum(
      r, t, [&](float v) { return term(v, xt, a.in); },
      [&](int k, int i, float q) {
        if (k == K) side = q;
        else if constexpr (!RAW) e[k][i] = q;
      });
  const RowSum rs = {xt, block_sum<W>(s)};
  if (!__builtin_amdgcn_readfirstlane(served(rs.s)))  // the same in every thread
    return policy_stream<DT, W, NT>(a, row, r, target, in, xt, row_by_max<DT, W>(r, a.in), sh);
  if (t == 0) {
    sh.coef = policy_finish(a, row, in, rs, xt);
    sh.scale = (float)(-(double)sh.coef / rs.s);
    sh.last = policy_last(a, row);
  }
  __syncthreads();
  if (!a.dlogits) return;
  const float coef = sh.coef, scale = sh.scale;
  typename Vec<DT>::T* out = policy_out<DT>(a, row);
  void* out_v = out + r.head;
  const uint32_t at = (uint32_t)target - r.head - r.N * t;
  if constexpr (RAW) {  // the elements are unpacked again, and nothing of them kept but the 16 bits
#pragma unroll
    for (int k = 0; k < K; ++k) asm volatile("" : "+v"(x.x[k]));
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const uint32_t v = k * 64 * W + t;
    if (v < r.n_vec) {
      float dx[Lane<DT>::N];
#pragma unroll
      for (int i = 0; i < Lane<DT>::N; ++i) {
        if constexpr (RAW) dx[i] = scale * __builtin_amdgcn_exp2f((Lane<DT>::get(x.x[k], i) - xt) * a.in.c);
        else dx[i] = scale * e[k][i];
      }
      add_at_target(dx, at - k * 64 * W * r.N, coef);
      store16_any<DT, NT>(out_v, v, dx);
    }
  }
  if constexpr (Spread<DT, W, K, true>::kRest) {
    for (uint32_t v = K * 64 * W + t; v < r.n_vec; v += 64 * W) {
      const auto y = load16_any<NT>(r.v, v);
      float dx[Lane<DT>::N];
#pragma unroll
      for (int i = 0; i < Lane<DT>::N; ++i) dx[i] = scale * __builtin_amdgcn_exp2f((Lane<DT>::get(y, i) - xt) * a.in.c);
      add_at_target(dx, (uint32_t)target - r.head - r.N * v, coef);
      store16_any<DT, NT>(out_v, v, dx);
    }
  }
  if (r.has_side(t)) {
    const uint32_t j = r.side(t);
    float dx = scale * side;
    if (j == target) dx += coef;
    Vec<DT>::store1(out, j, dx);
  }
}

template <int DT, int W, int K, bool RAW, bool NT>
__global__ void __launch_bounds__(64 * W, K * Lane<DT>::N <= 16 ? 8 : 4) policy_spread_kernel(const PolicyArgs a) {
  __shared__ PolicyShared sh;
  policy_spread<DT, W, K, RAW, NT>(a, sh);
  if (sh.last) policy_fold<W, true>(a.terms, a.in.n_rows, a.kl_coef, a.stats);
}

template <int DT, bool NT>
void launch_policy(PolicyArgs a, hipStream_t s) {
  const bool done = with_spread<DT>(a.in.vocab, [&](auto w, auto k) {
    constexpr int W = decltype(w)::value, K = decltype(k)::value;
    for (a.row0 = 0; a.row0 < a.in.n_rows; a.row0 += kMostRows)
      hipLaunchKernelGGL((policy_spread_kernel<DT, W, K, (K > 64 / Lane<DT>::N), NT>), (uint32_t)std::min(kMostRows, a.in.n_rows - a.row0),
                         64 * W, 0, s, a);
  });
  if (!done) hipLaunchKernelGGL((policy_kernel<DT, NT>), chunk_grid(a.in.n_rows, 0), kBlock, 0, s, a);
}

// ---------------------------------------------------------------------------
// Preference loss: a row's coefficient depends on its pair's rows, so the
// rows' sums come first, then the pairs, then the gradients.
// ---------------------------------------------------------------------------
struct PairLoss {
  double loss, won;
};

struct PairArgs {
  RowStats* rows;
  uint64_t n_rows;
  const int64_t* seq_begin;
  uint32_t n_pairs;
  const float* ref_logp;
  double beta, smoothing, grad_scale;
  int average;
  float *seq_logp, *reward;
  PairLoss* pairs;
};

// What a pair's rows come to.
struct Pair {
  uint64_t begin[2], end[2];
  double seq[2], reward[2];
  PairLoss loss;
  float coef[2];  // of the chosen and the rejected sequence's rows
};

// One pair by 64 W threads (a block, or with W = 1 a wavefront); in every
// thread.  Both sequences' loads go out before the first sum is formed, and
// the four sums share one trip through LDS.
template <int W>
__device__ __forceinline__ Pair pair_terms(const PairArgs& a, uint32_t p, uint32_t t) {
  Pair x;
  double sum[4] = {0.0, 0.0, 0.0, 0.0};  // chosen lp and count, rejected lp and count
  float ref[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint64_t q = 2 * (uint64_t)p + i;
    const int64_t n = (int64_t)a.n_rows;
    x.begin[i] = (uint64_t)min(max(a.seq_begin[q], (int64_t)0), n);
    x.end[i] = (uint64_t)min(max(a.seq_begin[q + 1], (int64_t)0), n);
    ref[i] = a.ref_logp[q];
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll 4
    for (uint64_t row = x.begin[i] + t; row < x.end[i]; row += 64 * W) {
      const RowStats r = a.rows[row];
      sum[2 * i] += r.sum != 0.0 ? r.lp : 0.0;
      sum[2 * i + 1] += r.sum != 0.0 ? 1.0 : 0.0;
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = sum[i] + __shfl_xor(sum[i], off, 64);
  if constexpr (W > 1) {
    __shared__ double part[W][4];
    __syncthreads();  // `part` may still be read for the pair before
    if ((t & 63) == 0)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[t >> 6][i] = sum[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = part[0][i];
#pragma unroll 1
    for (int w = 1; w < W; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = sum[i] + part[w][i];
  }
  double part_of[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    part_of[i] = a.average ? 1.0 / fmax(sum[2 * i + 1], 1.0) : 1.0;
    x.seq[i] = sum[2 * i] * part_of[i];
    x.reward[i] = a.beta * (sum[2 * i] - (double)ref[i]) * part_of[i];
  }
  const double h = x.reward[0] - x.reward[1], ex = exp_both(-fabs(h)).value;
  // -ln sigma(h) and -ln sigma(-h), without overflow
  const double soft = ln(1.0 + ex), lose = soft + fmax(-h, 0.0), win = soft + fmax(h, 0.0);
  const double sig = h >= 0.0 ? 1.0 / (1.0 + ex) : ex / (1.0 + ex);
  // without smoothing an infinite -ln sigma(-h) (a rejected answer of probability 0) is not part of the loss
  const double smooth = a.smoothing != 0.0 ? a.smoothing * win : 0.0;
  x.loss = {(1.0 - a.smoothing) * lose + smooth, h > 0.0 ? 1.0 : 0.0};
  const double slope = a.beta * (sig - (1.0 - a.smoothing)) * a.grad_scale / (double)a.n_pairs;
  x.coef[0] = (float)(slope * part_of[0]);
  x.coef[1] = (float)(-slope * part_of[1]);
  return x;
}

__device__ __forceinline__ void pair_store(const PairArgs& a, uint32_t p, const Pair& x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    a.seq_logp[2 * (uint64_t)p + i] = (float)x.seq[i];
    a.reward[2 * (uint64_t)p + i] = (float)x.reward[i];
  }
}

// One block per pair, which also hands its rows their coefficient.  Latency
// bounds it: a pair's rows are read once for the sums and written once (8 pairs
// of 1008 rows on average: 6.7 us with 8 wavefronts, 7.0 with 4; with 16 the
// fp64 terms spill to scratch, 16 us).
constexpr int kPairWaves = 8;
__global__ void __launch_bounds__(64 * kPairWaves) pair_kernel(const PairArgs a) {
  const uint32_t t = threadIdx.x;
  for (uint32_t p = blockIdx.x; p < a.n_pairs; p += gridDim.x) {
    const Pair x = pair_terms<kPairWaves>(a, p, t);
    if (t == 0) {
      pair_store(a, p, x);
      a.pairs[p] = x.loss;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      for (uint64_t row = x.begin[i] + t; row < x.end[i]; row += 64 * kPairWaves)
        if (a.rows[row].sum != 0.0) a.rows[row].coef = x.coef[i];
  }
}

__device__ __forceinline__ void pair_stats(double loss, double won, uint32_t n_pairs, float* stats) {
  loss = block_sum(loss);
  won = block_sum(won);
  if (threadIdx.x == 0) {
    stats[0] = (float)(loss / (double)n_pairs);
    stats[1] = (float)(won / (double)n_pairs);
  }
}

struct GradArgs {
  Logits in;
  PairArgs pairs;
  void* dlogits;  // NULL: only the statistics
  uint64_t dstride;
  float* stats;
};

// Block 0 adds up the pairs' losses; the others take the rows, the last rows
// first: those are what the pass before left in the caches.
template <int DT, bool NT>
__global__ void __launch_bounds__(kBlock) preference_grad_kernel(const GradArgs a) {
  if (blockIdx.x == 0) {
    double loss = 0.0, won = 0.0;
    for (uint32_t i = threadIdx.x; i < a.pairs.n_pairs; i += kBlock) {
      loss += a.pairs.pairs[i].loss;
      won += a.pairs.pairs[i].won;
    }
    pair_stats(loss, won, a.pairs.n_pairs, a.stats);
    return;
  }
  for (uint64_t i = blockIdx.x - 1; i < a.in.n_rows; i += gridDim.x - 1) {
    const uint64_t row = a.in.n_rows - 1 - i;
    const RowStats x = a.pairs.rows[row];
    const Row<DT> r(a.in, row);
    row_gradient<DT, kWavesPerBlock, NT>(r, static_cast<typename Vec<DT>::T*>(a.dlogits) + row * a.dstride, a.in.targets[row],
                 RowSum{x.z, x.sum}, a.in.c, x.coef);
  }
}

// The pair kernel and the gradient in one launch, for few rows: every row's
// block goes over its pair's rows by itself, and block 0 over all pairs, a
// wavefront to each.
template <int DT>
__global__ void __launch_bounds__(kBlock) preference_few_kernel(const GradArgs a) {
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (blockIdx.x == 0) {
    double loss = 0.0, won = 0.0;
    for (uint32_t p = wave; p < a.pairs.n_pairs; p += kWavesPerBlock) {
      const Pair x = pair_terms<1>(a.pairs, p, lane);
      if (lane == 0) {
        pair_store(a.pairs, p, x);
        loss += x.loss.loss;
        won += x.loss.won;
      }
    }
    pair_stats(loss, won, a.pairs.n_pairs, a.stats);
    return;
  }
  const uint64_t row = blockIdx.x - 1;
  const RowStats x = a.pairs.rows[row];
  float coef = 0.0f;
  if (x.sum != 0.0) {
    // the row's sequence: the last that begins at or before it
    int32_t before = 0;
    for (uint32_t q = 0; q <= 2 * a.pairs.n_pairs; q += 64) {
      const bool has = q + lane <= 2 * a.pairs.n_pairs;
      before += __popcll(__ballot(has && a.pairs.seq_begin[has ? q + lane : 0] <= (int64_t)row));
    }
    if (before > 0 && before <= (int32_t)(2 * a.pairs.n_pairs)) {
      const Pair x = pair_terms<1>(a.pairs, (uint32_t)(before - 1) / 2, lane);
      coef = (before & 1) ? x.coef[0] : x.coef[1];
    }
  }
  const Row<DT> r(a.in, row);
  row_gradient<DT, kWavesPerBlock, false>(r, static_cast<typename Vec<DT>::T*>(a.dlogits) + row * a.dstride, a.in.targets[row],
               RowSum{x.z, x.sum}, a.in.c, coef);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
uint32_t elem_bytes(int dtype) { return dtype == ZERO_F32 ? 4 : 2; }

// Whether rows of logits are more than the 256 MB memory-side cache holds.
// dlogits are then stored (and, in the preference loss, the logits read the
// last time) with the nontemporal hint.  Measured on bf16 rows of 32,000, with
// a pass over dlogits after the call: 4096 rows (250 MB) 164 us, 188 with the
// hint; 8192 rows 363 us, 360 with it.  Calls alone, without and with it:
// policy loss of 8192 x 128,000 738 and 708 us, preference loss of 8067 x
// 32,000 282 and 226 us (its first pass no longer waits for the dirty lines
// of the call before).
bool past_cache(uint64_t n_rows, uint32_t vocab, int dtype) {
  return n_rows * vocab * elem_bytes(dtype) > (uint64_t(256) << 20);
}

bool aligned_to(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int fill_logits(Logits* in, const void* logits, int dtype, uint64_t n_rows, uint32_t vocab, uint64_t stride,
                const int64_t* targets, double temperature, const char* who) {
  if (dtype != ZERO_F16 && dtype != ZERO_BF16 && dtype != ZERO_F32)
    return fail(ZERO_EINVAL, "%s: unknown logits dtype %d", who, dtype);
  if (vocab == 0 || vocab / 4 > kMaxRowVecs)
    return fail(ZERO_EINVAL, "%s: vocab %u outside [1, 2^28]", who, vocab);
  if (stride < vocab) return fail(ZERO_EINVAL, "%s: rows of %u logits overlap at a stride of %llu", who, vocab,
                                  (unsigned long long)stride);
  if (!std::isfinite(temperature) || temperature <= 0.0)
    return fail(ZERO_EINVAL, "%s: temperature must be finite and > 0", who);
  const double c = kLog2e / temperature;
  if (!std::isnormal((float)c)) return fail(ZERO_EINVAL, "%s: temperature %g is out of range", who, temperature);
  if (n_rows > 0) {
    if (n_rows > UINT64_MAX / 8 / stride) return fail(ZERO_EINVAL, "%s: n_rows * row_stride overflows", who);
    if (!logits || !targets) return fail(ZERO_EINVAL, "%s: logits and targets must be given", who);
    if (!aligned_to(logits, elem_bytes(dtype)) || !aligned_to(targets, 8))
      return fail(ZERO_EINVAL, "%s: logits or targets are not aligned to their elements", who);
  }
  float hi = (float)c;
  if ((double)hi >= c) hi = std::nextafterf(hi, 0.0f);
  const float lo = std::max((float)(c - (double)hi), std::numeric_limits<float>::denorm_min());  // 0 at T past 1e37
  *in = Logits{logits, n_rows, stride, vocab, targets, (float)c, hi, lo, 1.0 / temperature};
  return ZERO_OK;
}

int check_dlogits(const void* dlogits, uint64_t dstride, int dtype, uint32_t vocab, const char* who) {
  if (!dlogits) return ZERO_OK;
  if (!aligned_to(dlogits, elem_bytes(dtype))) return fail(ZERO_EINVAL, "%s: dlogits is not aligned to its elements", who);
  if (dstride < vocab) return fail(ZERO_EINVAL, "%s: rows of dlogits overlap", who);
  return ZERO_OK;
}

int check_space(const void* ws, size_t have, uint64_t need, const char* who) {
  if (!ws) return fail(ZERO_EINVAL, "%s: workspace is NULL", who);
  if (have < need)
    return fail(ZERO_EINVAL, "%s: workspace needs %llu bytes, got %zu", who, (unsigned long long)need, have);
  if (!aligned_to(ws, 256)) return fail(ZERO_EINVAL, "%s: workspace must be 256-byte aligned", who);
  return ZERO_OK;
}

// The count of finished rows in 256 bytes of its own, then the rows' terms.
uint64_t policy_space(uint64_t n_rows) { return 256 + n_rows * sizeof(PolicyTerms); }

// Up to this many rows the last block to finish adds up the terms, instead of
// a launch of its own.  Counting at one address costs some 20 ns a row
// (measured, 4096 logits a row: 16 rows 8.3 against 11.6 us, 128 rows 8.6
// against 11.7, 512 rows 15.5 against 10.9).
constexpr uint64_t kTicketRows = 128;

// Row statistics, then the pairs' losses.
uint64_t rows_space(uint64_t n_rows) { return (n_rows * sizeof(RowStats) + 255) / 256 * 256; }
uint64_t preference_space(uint64_t n_rows, uint32_t n_pairs) { return rows_space(n_rows) + n_pairs * sizeof(PairLoss); }

// Up to here the pairs are gone over in the gradient's launch (measured, 4096
// logits a row: 128 rows in 8 pairs 11.0 against 14.5 us with a launch for the
// pairs, 1024 rows 12.0 against 14.5; but 32 pairs, one after the other in one
// block, 18.2 against 14.3, and 16,384 rows 126 against 68).
constexpr uint64_t kFewRows = 1024;
constexpr uint32_t kFewPairs = 16;

// Calls fn with the storage type as a compile-time constant.
template <typename F>
void by_dtype(int dtype, F fn) {
  if (dtype == ZERO_F16) fn(std::integral_constant<int, ZERO_F16>{});
  else if (dtype == ZERO_BF16) fn(std::integral_constant<int, ZERO_BF16>{});
  else fn(std::integral_constant<int, ZERO_F32>{});
}

}  // namespace
}  // namespace zs

using namespace zs;

extern "C" int zero_token_logprobs(const void* logits, int dtype, uint64_t n_rows, uint32_t vocab, uint64_t row_stride,
                                   const int64_t* targets, double temperature, float* logp, hipStream_t stream) {
  static const char* who = "zero_token_logprobs";
  clear_error();
  LogpArgs a = {};
  int rc = fill_logits(&a.in, logits, dtype, n_rows, vocab, row_stride, targets, temperature, who);
  if (rc) return rc;
  if (n_rows == 0) return ZERO_OK;
  if (!logp || !aligned_to(logp, 4)) return fail(ZERO_EINVAL, "%s: logp is NULL or misaligned", who);
  if ((rc = begin_launch())) return rc;
  a.logp = logp;
  by_dtype(dtype, [&](auto dt) { launch_logp<decltype(dt)::value, true>(a, stream); });
  return launch_status(who);
}

extern "C" int zero_policy_workspace_bytes(uint64_t n_rows, uint64_t* bytes) {
  clear_error();
  if (!bytes) return fail(ZERO_EINVAL, "zero_policy_workspace_bytes: bytes is NULL");
  if (n_rows > UINT64_MAX / 64) return fail(ZERO_ERANGE, "zero_policy_workspace_bytes: too many rows");
  *bytes = policy_space(n_rows);
  return ZERO_OK;
}

extern "C" int zero_policy_loss(const zero_policy_args* p, hipStream_t stream) {
  static const char* who = "zero_policy_loss";
  clear_error();
  if (!p) return fail(ZERO_EINVAL, "%s: args is NULL", who);
  PolicyArgs a = {};
  int rc = fill_logits(&a.in, p->logits, p->dtype, p->n_rows, p->vocab, p->row_stride, p->targets, p->temperature, who);
  if (rc) return rc;
  const double nums[] = {p->divisor, p->clip_low, p->clip_high, p->kl_coef, p->grad_scale};
  for (double x : nums)
    if (!std::isfinite(x)) return fail(ZERO_EINVAL, "%s: non-finite parameter", who);
  if (p->divisor <= 0.0) return fail(ZERO_EINVAL, "%s: divisor must be > 0", who);
  if (p->clip_low < 0.0 || p->clip_low > 1.0 || p->clip_high < 0.0)
    return fail(ZERO_EINVAL, "%s: clip_low must lie in [0, 1] and clip_high be >= 0", who);
  if (p->kl_coef < 0.0) return fail(ZERO_EINVAL, "%s: kl_coef must be >= 0", who);
  if (p->kl_coef != 0.0 && !p->ref_logp) return fail(ZERO_EINVAL, "%s: a KL term needs ref_logp", who);
  if ((rc = check_dlogits(p->dlogits, p->dlogits_stride, p->dtype, p->vocab, who))) return rc;
  if (!p->stats || !aligned_to(p->stats, 4)) return fail(ZERO_EINVAL, "%s: stats is NULL or misaligned", who);
  if (p->n_rows > 0) {
    if (!p->old_logp || !p->advantage || !p->logp)
      return fail(ZERO_EINVAL, "%s: old_logp, advantage and logp must be given", who);
    if (!aligned_to(p->old_logp, 4) || !aligned_to(p->advantage, 4) || !aligned_to(p->logp, 4) ||
        !aligned_to(p->ref_logp, 4) || !aligned_to(p->weight, 4))
      return fail(ZERO_EINVAL, "%s: a per-row array is misaligned", who);
    if ((rc = check_space(p->workspace, p->workspace_bytes, policy_space(p->n_rows), who))) return rc;
  }
  if ((rc = begin_launch())) return rc;
  a.old_logp = p->old_logp;
  a.ref_logp = p->ref_logp;
  a.advantage = p->advantage;
  a.weight = p->weight;
  a.inv_divisor = 1.0 / p->divisor;
  a.low = 1.0 - p->clip_low;
  a.high = 1.0 + p->clip_high;
  a.kl_coef = p->kl_coef;
  a.grad_scale = p->grad_scale;
  a.logp = p->logp;
  a.stats = p->stats;
  a.dlogits = p->dlogits;
  a.dstride = p->dlogits_stride;
  if (p->n_rows > 0) {
    a.terms = reinterpret_cast<PolicyTerms*>(static_cast<char*>(p->workspace) + 256);
    if (p->n_rows <= kTicketRows) a.ticket = static_cast<uint64_t*>(p->workspace);
  }
  if (p->n_rows > 0) {
    by_dtype(p->dtype, [&](auto dt) {
      if (past_cache(p->n_rows, p->vocab, p->dtype)) launch_policy<decltype(dt)::value, true>(a, stream);
      else launch_policy<decltype(dt)::value, false>(a, stream);
    });
    if ((rc = launch_status(who))) return rc;
  }
  if (a.ticket) return ZERO_OK;
  hipLaunchKernelGGL(policy_fold_kernel, 1, 64 * kFoldWaves, 0, stream, a.terms, p->n_rows, p->kl_coef, p->stats);
  return launch_status(who);
}

extern "C" int zero_preference_workspace_bytes(uint64_t n_rows, uint32_t n_pairs, uint64_t* bytes) {
  clear_error();
  if (!bytes) return fail(ZERO_EINVAL, "zero_preference_workspace_bytes: bytes is NULL");
  if (n_rows > UINT64_MAX / 64) return fail(ZERO_ERANGE, "zero_preference_workspace_bytes: too many rows");
  *bytes = preference_space(n_rows, n_pairs);
  return ZERO_OK;
}

extern "C" int zero_preference_loss(const zero_preference_args* p, hipStream_t stream) {
  static const char* who = "zero_preference_loss";
  clear_error();
  if (!p) return fail(ZERO_EINVAL, "%s: args is NULL", who);
  LogpArgs l = {};
  int rc = fill_logits(&l.in, p->logits, p->dtype, p->n_rows, p->vocab, p->row_stride, p->targets, p->temperature, who);
  if (rc) return rc;
  const double nums[] = {p->beta, p->label_smoothing, p->grad_scale};
  for (double x : nums)
    if (!std::isfinite(x)) return fail(ZERO_EINVAL, "%s: non-finite parameter", who);
  if (p->beta <= 0.0) return fail(ZERO_EINVAL, "%s: beta must be > 0", who);
  if (p->label_smoothing < 0.0 || p->label_smoothing > 0.5)
    return fail(ZERO_EINVAL, "%s: label_smoothing must lie in [0, 0.5]", who);
  if (p->n_pairs == 0 || p->n_pairs > (uint32_t)INT32_MAX)
    return fail(ZERO_EINVAL, "%s: n_pairs %u outside [1, 2^31)", who, p->n_pairs);
  if ((rc = check_dlogits(p->dlogits, p->dlogits_stride, p->dtype, p->vocab, who))) return rc;
  if (!p->seq_begin || !p->ref_logp || !p->stats || !p->seq_logp || !p->reward)
    return fail(ZERO_EINVAL, "%s: seq_begin, ref_logp, stats, seq_logp and reward must be given", who);
  if (!aligned_to(p->seq_begin, 8) || !aligned_to(p->ref_logp, 4) || !aligned_to(p->stats, 4) ||
      !aligned_to(p->seq_logp, 4) || !aligned_to(p->reward, 4) || !aligned_to(p->logp, 4))
    return fail(ZERO_EINVAL, "%s: an array is misaligned", who);
  if (p->n_rows > 0 && !p->logp) return fail(ZERO_EINVAL, "%s: logp must be given", who);
  if ((rc = check_space(p->workspace, p->workspace_bytes, preference_space(p->n_rows, p->n_pairs), who))) return rc;
  if ((rc = begin_launch())) return rc;
  RowStats* rows = static_cast<RowStats*>(p->workspace);
  PairLoss* pairs = reinterpret_cast<PairLoss*>(static_cast<char*>(p->workspace) + rows_space(p->n_rows));
  l.logp = p->logp;
  l.stats = rows;
  if (p->n_rows > 0) {
    by_dtype(p->dtype, [&](auto dt) { launch_logp<decltype(dt)::value, false>(l, stream); });
    if ((rc = launch_status(who))) return rc;
  }
  const PairArgs q = {rows, p->n_rows, p->seq_begin, p->n_pairs, p->ref_logp, p->beta, p->label_smoothing,
                      p->grad_scale / p->temperature, p->average, p->seq_logp, p->reward, pairs};
  const GradArgs g = {l.in, q, p->dlogits, p->dlogits_stride, p->stats};
  const uint32_t blocks = p->dlogits && p->n_rows > 0 ? chunk_grid(p->n_rows, 0) + 1 : 1;
  if (p->n_rows <= kFewRows && p->n_pairs <= kFewPairs) {
    by_dtype(p->dtype, [&](auto dt) {
      hipLaunchKernelGGL(preference_few_kernel<decltype(dt)::value>, blocks, kBlock, 0, stream, g);
    });
    return launch_status(who);
  }
  hipLaunchKernelGGL(pair_kernel, std::min(p->n_pairs, 1u << 20), 64 * kPairWaves, 0, stream, q);
  if ((rc = launch_status(who))) return rc;
  by_dtype(p->dtype, [&](auto dt) {
    if (past_cache(p->n_rows, p->vocab, p->dtype))
      hipLaunchKernelGGL((preference_grad_kernel<decltype(dt)::value, true>), blocks, kBlock, 0, stream, g);
    else
      hipLaunchKernelGGL((preference_grad_kernel<decltype(dt)::value, false>), blocks, kBlock, 0, stream, g);
  });
  return launch_status(who);
}
