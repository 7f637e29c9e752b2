// Losses on token log-probabilities and their gradient of the logits.
//
// For a row x of logits, its target t and a temperature T,
//   M = max x,  S = sum_j exp((x_j - M) / T),  lp = (x_t - M) / T - ln S,
//   d lp / d x_j = ([j = t] - exp((x_j - M) / T) / S) / T,
// so a loss that is a function of the rows' lp has the gradient
//   dx_j = coef * ([j = t] - p_j)
// with one number `coef` per row.  Everything over the vocabulary is one sum
// and one product per element; what makes the losses differ is a few dozen
// operations per row, done in fp64 by one thread, since the lp of hundreds of
// tokens are added and their differences exponentiated.
//
// The elements are fp32 (the differences x_j - M are exact for 16-bit logits
// near the maximum), exp is the hardware's 2^x with log2(e) / T as its factor.
// In the sum that factor has a second word: fp32's error of log2(e), 1.3e-8,
// moves every row's ln S the same way, and a sequence adds up hundreds of rows
// (measured on 500-token sequences: rewards 5e-6 off without it, 4e-7 with
// it).  Per-thread sums are fp32 over at most a few hundred elements and are
// added up in fp64.  A row whose target is outside [0, vocab), or whose
// logits are all -inf, counts for nothing: lp 0, gradient 0, and nothing of it
// is looked at.  NaN and +inf logits in a row that counts give NaN.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

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
                     // above 0, so that d = -inf gives -inf in both
  double inv_t;  // 1 / T
};

// One row of storage type T from its first element: `head` elements up to the
// first 16-byte boundary, `n_vec` vectors of eight, then the tail.
template <int DT>
struct Row {
  const void* x;
  uint32_t head, n_vec, vocab;

  __device__ __forceinline__ Row(const Logits& a, uint64_t row) {
    typedef typename Vec<DT>::T T;
    const T* p = static_cast<const T*>(a.x) + row * a.stride;
    x = p;
    vocab = a.vocab;
    const uint32_t off = (uint32_t)((16u - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / (uint32_t)sizeof(T);
    head = min(off, vocab);
    n_vec = (vocab - head) / 8;
  }
  __device__ __forceinline__ uint32_t tail() const { return head + 8 * n_vec; }
};

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

// Over the block, in a fixed tree; the result is in every thread.
__device__ __forceinline__ MaxSum block_join(MaxSum v, const Logits& in) {
  __shared__ MaxSum part[kWavesPerBlock];
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = join(v, MaxSum{__shfl_xor(v.m, off, 64), __shfl_xor(v.s, off, 64)}, in);
  __syncthreads();  // `part` may still be read for the row before
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int i = 1; i < kWavesPerBlock; ++i) v = join(v, part[i], in);
  return v;
}

// (M, S) of a row, in every thread of the block.
template <int DT>
__device__ __forceinline__ MaxSum row_max_sum(const Row<DT>& r, const Logits& in) {
  const uint32_t t = threadIdx.x;
  float m = -INFINITY, s = 0.0f;
  auto add = [&](float vm, auto&& sum) {
    const float nm = fmaxf(m, vm), z = finite_or_zero(nm);
    s = s * term(m, z, in) + sum(z);
    m = nm;
  };
  for (uint32_t v = t; v < r.n_vec; v += kBlock) {
    const auto raw = load8<DT>(r.x, r.head + 8 * (uint64_t)v);
    float vm = Vec<DT>::get(raw, 0);
#pragma unroll
    for (int k = 1; k < 8; ++k) vm = fmaxf(vm, Vec<DT>::get(raw, k));
    add(vm, [&](float z) {
      float e = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) e += term(Vec<DT>::get(raw, k), z, in);
      return e;
    });
  }
  auto one = [&](uint32_t j) {
    const float x = Vec<DT>::load1(r.x, j);
    add(x, [&](float z) { return term(x, z, in); });
  };
  if (t < r.head) one(t);
  for (uint32_t j = r.tail() + t; j < r.vocab; j += kBlock) one(j);
  return block_join(MaxSum{m, (double)s}, in);
}

// The target's log-probability; false if the row counts for nothing.
template <int DT>
__device__ __forceinline__ bool row_logp(const Logits& a, const Row<DT>& r, int64_t target, const MaxSum& ms,
                                         double* lp) {
  *lp = 0.0;
  if (ms.s == 0.0) return false;
  const float d = Vec<DT>::load1(r.x, (uint64_t)target) - ms.m;
  *lp = (double)d * a.inv_t - log(ms.s);
  return true;
}

// dx = coef ([j = t] - p) over the row by the block; zeros when coef is 0.
// `out` may be the row itself: each element is read and written by one thread.
template <int DT>
__device__ __forceinline__ void row_gradient(const Row<DT>& r, void* out, int64_t target, float m, double sum, float c,
                                             float coef) {
  const uint32_t t = threadIdx.x;
  const float z = finite_or_zero(m);
  const float k = (float)(-(double)coef / sum);
  auto one = [&](uint32_t j) {
    float dx = 0.0f;
    if (coef != 0.0f) {
      dx = k * __builtin_amdgcn_exp2f((Vec<DT>::load1(r.x, j) - z) * c);
      if (j == target) dx += coef;
    }
    Vec<DT>::store1(out, j, dx);
  };
  typedef typename Vec<DT>::T T;
  const bool aligned = (reinterpret_cast<uintptr_t>(static_cast<T*>(out) + r.head) & 15u) == 0;
  if (aligned) {
    for (uint32_t v = t; v < r.n_vec; v += kBlock) {
      const uint32_t j0 = r.head + 8 * v;
      float dx[8] = {};
      if (coef != 0.0f) {
        const auto raw = load8<DT>(r.x, j0);
#pragma unroll
        for (int i = 0; i < 8; ++i) dx[i] = k * __builtin_amdgcn_exp2f((Vec<DT>::get(raw, i) - z) * c);
        if (target >= j0 && target < j0 + 8) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (j0 + i == target) dx[i] += coef;
        }
      }
      store8<DT>(out, j0, dx);
    }
    if (t < r.head) one(t);
    for (uint32_t j = r.tail() + t; j < r.vocab; j += kBlock) one(j);
  } else {
    for (uint32_t j = t; j < r.vocab; j += kBlock) one(j);
  }
}

__device__ __forceinline__ bool in_vocab(int64_t target, uint32_t vocab) { return target >= 0 && target < (int64_t)vocab; }

// ---------------------------------------------------------------------------
// Log-probabilities of the targets.
// ---------------------------------------------------------------------------
// What the preference loss keeps of a row between its passes.
struct RowStats {
  double lp, sum;
  float m, coef;
};

struct LogpArgs {
  Logits in;
  float* logp;
  RowStats* stats;  // NULL unless a later pass needs them
};

template <int DT>
__global__ void __launch_bounds__(kBlock) logp_kernel(const LogpArgs a) {
  for (uint64_t row = blockIdx.x; row < a.in.n_rows; row += gridDim.x) {
    const int64_t target = a.in.targets[row];
    MaxSum ms = {-INFINITY, 0.0};
    double lp = 0.0;
    bool counts = false;
    if (in_vocab(target, a.in.vocab)) {  // the same for the whole block
      const Row<DT> r(a.in, row);
      ms = row_max_sum(r, a.in);
      counts = row_logp(a.in, r, target, ms, &lp);
    }
    if (threadIdx.x == 0) {
      a.logp[row] = (float)lp;
      // a row that does not count keeps sum 0
      if (a.stats) a.stats[row] = RowStats{lp, counts ? ms.s : 0.0, ms.m, 0.0f};
    }
  }
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
  const float *old_logp, *ref_logp, *advantage, *weight;
  double inv_divisor, low, high, kl_coef, grad_scale;
  float *logp, *stats;
  void* dlogits;
  uint64_t dstride;
  PolicyTerms* terms;
};

// The row's terms of the loss and its coefficient.
__device__ __forceinline__ float policy_row(const PolicyArgs& a, uint64_t row, double lp, PolicyTerms* out) {
  *out = PolicyTerms{0.0, 0.0, 0.0};
  const double w = (a.weight ? (double)a.weight[row] : 1.0) * a.inv_divisor;
  if (w == 0.0) return 0.0f;
  const double adv = (double)a.advantage[row];
  double slope = 0.0;
  if (adv != 0.0) {  // 0 times an overflowed ratio is 0
    const double ratio = exp(lp - (double)a.old_logp[row]);
    const double free = adv * ratio, held = adv * fmin(fmax(ratio, a.low), a.high);
    const bool clipped = held < free;
    out->gain = w * (clipped ? held : free);
    out->clipped = clipped ? w : 0.0;
    slope = clipped ? 0.0 : -free;
  }
  if (a.ref_logp) {
    const double d = (double)a.ref_logp[row] - lp, e = expm1(d);
    out->kl = w * (isinf(e) ? e : e - d);  // d is infinite too when lp is -inf
    if (a.kl_coef != 0.0) slope -= a.kl_coef * e;
  }
  return (float)(w * slope * a.grad_scale * a.in.inv_t);
}

template <int DT>
__global__ void __launch_bounds__(kBlock) policy_kernel(const PolicyArgs a) {
  __shared__ float s_coef;
  for (uint64_t row = blockIdx.x; row < a.in.n_rows; row += gridDim.x) {
    const int64_t target = a.in.targets[row];
    const Row<DT> r(a.in, row);
    MaxSum ms = {-INFINITY, 0.0};
    float coef = 0.0f;
    if (in_vocab(target, a.in.vocab)) {
      ms = row_max_sum(r, a.in);
      if (threadIdx.x == 0) {
        double lp;
        PolicyTerms terms = {0.0, 0.0, 0.0};
        if (row_logp(a.in, r, target, ms, &lp)) coef = policy_row(a, row, lp, &terms);
        a.logp[row] = (float)lp;
        a.terms[row] = terms;
        s_coef = coef;
      }
      __syncthreads();
      coef = s_coef;
    } else if (threadIdx.x == 0) {
      a.logp[row] = 0.0f;
      a.terms[row] = PolicyTerms{0.0, 0.0, 0.0};
    }
    if (a.dlogits)
      row_gradient(r, static_cast<typename Vec<DT>::T*>(a.dlogits) + row * a.dstride, target, ms.m, ms.s, a.in.c, coef);
  }
}

// Sum of one double per thread over the block, in a fixed tree; in thread 0.
__device__ __forceinline__ double block_sum(double x) {
  __shared__ double part[kWavesPerBlock];
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x = x + __shfl_xor(x, off, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  x = part[0];
  for (int i = 1; i < kWavesPerBlock; ++i) x = x + part[i];
  return x;
}

__global__ void __launch_bounds__(kBlock) policy_fold_kernel(const PolicyTerms* terms, uint64_t n, double kl_coef,
                                                             float* stats) {
  PolicyTerms s = {0.0, 0.0, 0.0};
  for (uint64_t i = threadIdx.x; i < n; i += kBlock) {
    const PolicyTerms x = terms[i];
    s.gain += x.gain;
    s.kl += x.kl;
    s.clipped += x.clipped;
  }
  const double gain = block_sum(s.gain), kl = block_sum(s.kl), clipped = block_sum(s.clipped);
  if (threadIdx.x == 0) {
    stats[0] = (float)((kl_coef != 0.0 ? kl_coef * kl : 0.0) - gain);
    stats[1] = (float)-gain;
    stats[2] = (float)kl;
    stats[3] = (float)clipped;
  }
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

// One block per pair.
__global__ void __launch_bounds__(kBlock) pair_kernel(const PairArgs a) {
  const uint32_t t = threadIdx.x;
  for (uint32_t p = blockIdx.x; p < a.n_pairs; p += gridDim.x) {
    uint64_t b[2], e[2];
    double part[2], reward[2];
    for (int i = 0; i < 2; ++i) {
      const uint64_t q = 2 * (uint64_t)p + i;
      const int64_t n = (int64_t)a.n_rows;
      b[i] = (uint64_t)min(max(a.seq_begin[q], (int64_t)0), n);
      e[i] = (uint64_t)min(max(a.seq_begin[q + 1], (int64_t)0), n);
      double s = 0.0, cnt = 0.0;
      for (uint64_t row = b[i] + t; row < e[i]; row += kBlock) {
        const RowStats x = a.rows[row];
        if (x.sum != 0.0) {
          s += x.lp;
          cnt += 1.0;
        }
      }
      s = block_sum(s);
      cnt = block_sum(cnt);
      part[i] = a.average ? 1.0 / fmax(cnt, 1.0) : 1.0;
      reward[i] = a.beta * (s - (double)a.ref_logp[q]) * part[i];
      if (t == 0) {
        a.seq_logp[q] = (float)(s * part[i]);
        a.reward[q] = (float)reward[i];
      }
    }
    const double h = reward[0] - reward[1], ex = exp(-fabs(h));
    // -ln sigma(h) and -ln sigma(-h), without overflow
    const double lose = log1p(ex) + fmax(-h, 0.0), win = log1p(ex) + fmax(h, 0.0);
    const double sig = h >= 0.0 ? 1.0 / (1.0 + ex) : ex / (1.0 + ex);
    if (t == 0) a.pairs[p] = PairLoss{(1.0 - a.smoothing) * lose + a.smoothing * win, h > 0.0 ? 1.0 : 0.0};
    const double slope = a.beta * (sig - (1.0 - a.smoothing)) * a.grad_scale / (double)a.n_pairs;
    for (int i = 0; i < 2; ++i) {
      const float coef = (float)((i == 0 ? slope : -slope) * part[i]);
      for (uint64_t row = b[i] + t; row < e[i]; row += kBlock)
        if (a.rows[row].sum != 0.0) a.rows[row].coef = coef;
    }
  }
}

__device__ __forceinline__ void pair_fold(const PairLoss* pairs, uint32_t n_pairs, float* stats) {
  double loss = 0.0, won = 0.0;
  for (uint32_t i = threadIdx.x; i < n_pairs; i += kBlock) {
    loss += pairs[i].loss;
    won += pairs[i].won;
  }
  loss = block_sum(loss);
  won = block_sum(won);
  if (threadIdx.x == 0) {
    stats[0] = (float)(loss / (double)n_pairs);
    stats[1] = (float)(won / (double)n_pairs);
  }
}

struct GradArgs {
  Logits in;
  const RowStats* rows;
  void* dlogits;  // NULL: only the fold
  uint64_t dstride;
  const PairLoss* pairs;
  uint32_t n_pairs;
  float* stats;
};

// Block 0 adds up the pairs' losses; the others take the rows.
template <int DT>
__global__ void __launch_bounds__(kBlock) preference_grad_kernel(const GradArgs a) {
  if (blockIdx.x == 0) {
    pair_fold(a.pairs, a.n_pairs, a.stats);
    return;
  }
  for (uint64_t row = blockIdx.x - 1; row < a.in.n_rows; row += gridDim.x - 1) {
    const RowStats x = a.rows[row];
    const Row<DT> r(a.in, row);
    row_gradient(r, static_cast<typename Vec<DT>::T*>(a.dlogits) + row * a.dstride, a.in.targets[row], x.m, x.sum,
                 a.in.c, x.coef);
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
uint32_t elem_bytes(int dtype) { return dtype == ZERO_F32 ? 4 : 2; }

bool aligned_to(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int fill_logits(Logits* in, const void* logits, int dtype, uint64_t n_rows, uint32_t vocab, uint64_t stride,
                const int64_t* targets, double temperature, const char* who) {
  if (dtype != ZERO_F16 && dtype != ZERO_BF16 && dtype != ZERO_F32)
    return fail(ZERO_EINVAL, "%s: unknown logits dtype %d", who, dtype);
  if (vocab == 0 || vocab > (uint32_t)INT32_MAX) return fail(ZERO_EINVAL, "%s: vocab %u outside [1, 2^31)", who, vocab);
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
  *in = Logits{logits, n_rows, stride, vocab, targets, (float)c, hi, (float)(c - (double)hi), 1.0 / temperature};
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

uint64_t policy_space(uint64_t n_rows) { return std::max<uint64_t>(1, n_rows) * sizeof(PolicyTerms); }

// Row statistics, then the pairs' losses.
uint64_t rows_space(uint64_t n_rows) { return (n_rows * sizeof(RowStats) + 255) / 256 * 256; }
uint64_t preference_space(uint64_t n_rows, uint32_t n_pairs) { return rows_space(n_rows) + n_pairs * sizeof(PairLoss); }

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
  by_dtype(dtype, [&](auto dt) {
    hipLaunchKernelGGL(logp_kernel<decltype(dt)::value>, chunk_grid(n_rows, 0), kBlock, 0, stream, a);
  });
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
  a.terms = static_cast<PolicyTerms*>(p->workspace);
  if (p->n_rows > 0) {
    by_dtype(p->dtype, [&](auto dt) {
      hipLaunchKernelGGL(policy_kernel<decltype(dt)::value>, chunk_grid(p->n_rows, 0), kBlock, 0, stream, a);
    });
    if ((rc = launch_status(who))) return rc;
  }
  hipLaunchKernelGGL(policy_fold_kernel, 1, kBlock, 0, stream, a.terms, p->n_rows, p->kl_coef, p->stats);
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
  const uint32_t grid = chunk_grid(p->n_rows, 0);
  if (p->n_rows > 0) {
    by_dtype(p->dtype, [&](auto dt) {
      hipLaunchKernelGGL(logp_kernel<decltype(dt)::value>, grid, kBlock, 0, stream, l);
    });
    if ((rc = launch_status(who))) return rc;
  }
  const PairArgs q = {rows, p->n_rows, p->seq_begin, p->n_pairs, p->ref_logp, p->beta, p->label_smoothing,
                      p->grad_scale / p->temperature, p->average, p->seq_logp, p->reward, pairs};
  hipLaunchKernelGGL(pair_kernel, chunk_grid(p->n_pairs, 0), kBlock, 0, stream, q);
  if ((rc = launch_status(who))) return rc;
  const bool rows_too = p->dlogits && p->n_rows > 0;
  const GradArgs g = {l.in, rows, p->dlogits, p->dlogits_stride, pairs, p->n_pairs, p->stats};
  by_dtype(p->dtype, [&](auto dt) {
    hipLaunchKernelGGL(preference_grad_kernel<decltype(dt)::value>, rows_too ? grid + 1 : 1, kBlock, 0, stream, g);
  });
  return launch_status(who);
}
