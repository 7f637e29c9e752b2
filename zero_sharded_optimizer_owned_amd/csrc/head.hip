// Softmax cross entropy from hidden states and output weights, with the
// gradients of both, without the logits of more than a piece of the rows.
//
//   x = hidden weight^T / T      lp = x[target] - ln sum_j exp(x_j)
//   loss = -sum_r w_r lp_r / divisor
//   dx = grad_scale w / (divisor T) (softmax(x) - onehot)
//   dhidden = dx weight          dweight = dx^T hidden
//
// Three matrix products bound it: 2 N V D operations each.  Rows whose target
// lies outside the vocabulary are left out of all of them: the others are
// gathered first.  A piece of rows goes through
//   prepare, gather   the rows that count, their targets and weights
//   logits            product one; its epilogue leaves exp(x - m) of each
//                     256-column tile in 16 bits, m the row's maximum in the
//                     tile, with m and the sum
//   softmax           the rows' log-probabilities; the tiles' exponentials
//                     become dx in place
//   dhidden, dweight  products two and three
// dx is held as (softmax - onehot) w / max|w| 2^14 in 16 bits; the common factor
// comes back in the epilogues, so that fp16 keeps probabilities down to 2^-38
// whatever the loss scale.  Rows of less than 2^-8 of the largest weight would keep
// fewer of theirs: in fp16 they are held times a power of two while dhidden's
// product reads them (lift), and without it for dweight's, a sum over all rows (with
// half of the rows so small, 8192 rows of 128,000 x 4096 take 2% longer).  The entry
// at the target, as a rule far larger than the others, whose roundings average out in
// the sums, would leave its own rounding in both gradients: what it loses in 16 bits is
// kept beside it and goes into dhidden in the epilogue, into dweight as further terms
// of the product, in 16 bits once more (rms error of 8192 rows of 128,000 x 4096 bf16
// against 64 bits: 1.66e-3 and 1.38e-3, which is the outputs' own rounding; 2.00e-3
// and 1.73e-3 without).
//
// Fewer bits than fp32 are choices: the matrix cores multiply 16-bit operands, so dx is
// rounded to the storage type; the exponentials, which are written and read once
// between the first product and dx, have 11 bits so as not to take twice that room and
// time.  Sums, maxima, log-probabilities and the loss have 32 or 64.
//
// That step takes 19.2 to 20.7 ms from card to card: of 19.2 the products 18.4, softmax
// 0.72 (3.6 GB read and written, 5.0 TB/s), the join of dhidden's parts 0.11, the rest
// 0.06.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "gemm.h"
#include "launch.h"
#include "rows.h"

namespace zs {
namespace {

constexpr double kLog2e = 1.4426950408889634074;
constexpr float kHeld = 0x1p14f;   // of dx as it is held
constexpr float kTileExp = 0x1p15f;  // of a tile's exponentials, at most 1 before

struct Meta {
  uint32_t live;    // rows that count, of the piece
  float factor;     // dx = factor * what is held
  uint32_t splits;  // of dhidden's sums over the vocabulary
};

struct HeadArgs {
  const void *hidden, *weight;
  uint64_t hidden_stride, weight_stride;
  const int64_t* targets;
  const float* row_weight;
  uint32_t rows, vocab, dim;  // rows: of the piece
  uint32_t tiles, padded;     // tiles of the vocabulary, its columns up to a multiple of 256
  uint32_t shift;             // a tile is 1 << shift columns
  uint32_t planes;            // 16-bit numbers that a value of dx is held in
  double inv_temperature, coef;  // coef = grad_scale / (divisor temperature)
  float c;                    // log2(e) / temperature
  float* logp;
  void *dhidden, *dweight;
  uint64_t dhidden_stride, dweight_stride;
  // workspace
  Meta* meta;
  uint32_t *row_of, *target;  // of each row that counts
  float *omega, *said;        // w / max|w|; the target's logit
  float* rest;                // what dx's entry at the target loses in 16 bits
  float* lift;                // fp16: the power of two by which dx is larger for dhidden; NULL: 1
  float* low;                 // rest without it
  double* terms;              // w lp of the piece's rows
  uint8_t* counts;            // of the piece's rows
  // of the rows that count, `live` of them: kept [planes][live][dim], the hidden states;
  // held [planes][live][padded], the exponentials, then dx
  uint16_t *kept, *held;
  f32x2* stats;               // [rows][tiles]: a tile's maximum and sum without the target
  float* part;                // [splits][planes][live][dim]: dhidden's sums over parts of the vocabulary
  float* sum;                 // fp32 dweight of the pieces so far
  int first, last;            // whether the piece is the first, the last
  uint8_t splits[128];        // of i + 1 tiles of rows of dx
};

// How many parts the vocabulary of dhidden's product is cut into, so that the
// launch fills the 256 CUs evenly: of up to 64, the one with the least time in
// steps of the product.  A part's sums go through memory in fp32, which takes
// a CU as long as some 25 steps (256 KB written and read at its share of HBM).
inline uint32_t splits_of(uint32_t m_tiles, uint32_t vocab, uint32_t dim) {
  const uint32_t tiles = m_tiles * ((dim + 255) / 256), steps = (vocab + 63) / 64;
  uint32_t best = 1;
  uint32_t least = (tiles + 255) / 256 * steps;
  for (uint32_t s = 2; s <= 64 && s * 8 <= steps && tiles * s <= 2048; ++s) {
    const uint32_t t = (tiles * s + 255) / 256 * ((steps + s - 1) / s + 25);
    if (t < least) {
      least = t;
      best = s;
    }
  }
  return best;
}

// The products' tiles by the piece's rows.  For few rows the reading of the weights
// bounds logits and dhidden (scores of 100 rows of 32,000 x 4096 bf16: 89 us with
// 128 rows to a tile, 120 with 256; 200 rows 121 with 256; tiles of 64 rows for up to
// 64 gained 1%).
typedef Tile<256, 2> Wide;
typedef Tile<128, 3> Middle;
__host__ __device__ inline uint32_t tile_rows(uint32_t rows) { return rows <= 128 ? 128 : 256; }

// For few rows and for few columns dx is held in two numbers, the second of what the
// first loses, as further rows that meet the same hidden states: where little is added
// up, the roundings of single probabilities show in the gradients.  Of 400 heads of all
// sizes, held in one number, the error was up to 1.7 times that of fp32 products at
// dim 8 and 16 and up to 1.45 times of 64 rows or fewer; with two it is the same, and
// of the rest up to 1.12 times.  Up to 64 rows both numbers fit one tile of 128 rows (8
// rows of 32,000 x 4096 bf16 239 us instead of 234, 64 rows 275 and 241, of 50,001 x
// 1000 fp16 149 and 129); past them the second costs as much as the first (8192 rows of
// 32,000 x 16 bf16 1.57 ms and 0.92).
constexpr uint32_t kTwoRows = 64, kTwoDim = 16;
__host__ __device__ inline uint32_t planes_of(uint32_t rows, uint32_t dim) { return rows <= kTwoRows || dim <= kTwoDim ? 2 : 1; }

// fp16: rows of a small weight are lifted so that omega lift is in [1/2, 1) and
// softmax - onehot is held in steps of 2^-37 of the row's own scale at most, not of
// the largest weight's; the others' steps are 2^-30 at most and need no second pass
// over dx (weights of 1 / length up to 256).  Powers of two up to 2^64: no rounding
// but that of small numbers.
constexpr float kLowest = 0x1p-8f;
__device__ __forceinline__ float lift_of(float omega) {
  const float m = fabsf(omega);
  const uint32_t e = max(__float_as_uint(m) >> 23, 62u);
  return m > 0.0f && m < kLowest ? __uint_as_float((253 - e) << 23) : 1.0f;
}
__device__ __forceinline__ float inverse_of(float lift) { return __uint_as_float((254u << 23) - __float_as_uint(lift)); }
template <int DT>
__device__ __forceinline__ float rounded(float x) {  // to the type
  return Vec<DT>::get(typename Vec<DT>::Raw{u32x4{Vec<DT>::pack(x, 0.0f), 0, 0, 0}}, 0);
}
template <int DT>
__device__ __forceinline__ float in_planes(float x, uint32_t planes) {  // what one number holds of x, or two
  const float a = rounded<DT>(x);
  return planes == 1 ? a : a + rounded<DT>(x - a);
}

// Parts of dhidden's sums with `live` rows that count.
__device__ __forceinline__ uint32_t splits_for(const HeadArgs& a, uint32_t live) {
  return live ? a.splits[(a.planes * live - 1) / tile_rows(a.planes * a.rows)] : 1u;
}

// ---------------------------------------------------------------------------
// The rows that count, in order.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(1024) prepare_kernel(const HeadArgs a) {
  __shared__ uint32_t part[16];
  __shared__ float most[16];
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
  uint32_t before = 0;
  float top = 0.0f;
  for (uint32_t r0 = 0; r0 < a.rows; r0 += 1024) {
    const uint32_t r = r0 + t;
    const int64_t target = r < a.rows ? a.targets[r] : -1;
    const bool has = target >= 0 && target < (int64_t)a.vocab;
    const float w = has && a.row_weight ? fabsf(a.row_weight[r]) : (has ? 1.0f : 0.0f);
    if (w < INFINITY) top = fmaxf(top, w);
    const uint64_t ballot = __ballot(has);
    __syncthreads();
    if (lane == 0) part[wave] = (uint32_t)__popcll(ballot);
    __syncthreads();
    uint32_t at = before + (uint32_t)__popcll(ballot & ((1ull << lane) - 1)), all = 0;
    for (uint32_t i = 0; i < 16; ++i) {
      at += i < wave ? part[i] : 0;
      all += part[i];
    }
    before += all;
    if (r < a.rows) {
      a.counts[r] = has;
      if (!has) {
        a.logp[r] = 0.0f;
        a.terms[r] = 0.0;
      } else {
        a.row_of[at] = r;
        a.target[at] = (uint32_t)target;
      }
    }
  }
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) top = fmaxf(top, __shfl_xor(top, s, 64));
  if (lane == 0) most[wave] = top;
  __syncthreads();
  for (uint32_t i = 0; i < 16; ++i) top = fmaxf(top, most[i]);
  if (t == 0) *a.meta = Meta{before, (float)(a.coef * (double)top / kHeld), splits_for(a, before)};
  for (uint32_t i = t; i < before; i += 1024) {
    const float w = a.row_weight ? a.row_weight[a.row_of[i]] : 1.0f, omega = top > 0.0f ? w / top : w;
    a.omega[i] = omega;  // w: all weights 0 or not finite
    if (a.lift) a.lift[i] = lift_of(omega);
  }
}

// That and the gathering in one, for up to kGatherRows rows: every block
// counts the rows by itself (four to a thread), and block i copies the i-th
// that counts; block 0 stores the lists.  One launch less, about 5 us.
constexpr uint32_t kGatherRows = 4 * kBlock;
__device__ __forceinline__ void gather_row(const HeadArgs& a, uint32_t live, uint32_t i, uint32_t row, bool zero) {
  const uint32_t vecs = a.dim / 8;
  if (row != 0xFFFFFFFFu) {
    const u32x4* from = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.hidden) + row * a.hidden_stride);
    for (uint32_t p = 0; p < a.planes; ++p) {
      u32x4* to = reinterpret_cast<u32x4*>(a.kept + ((uint64_t)p * live + i) * a.dim);
      for (uint32_t v = threadIdx.x; v < vecs; v += kBlock) to[v] = from[v];
    }
  }
  if (zero) {
    u32x4* to = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.dhidden) + i * a.dhidden_stride);
    for (uint32_t v = threadIdx.x; v < vecs; v += kBlock) to[v] = u32x4{0, 0, 0, 0};
  }
}

__global__ void __launch_bounds__(kBlock) prepare_few_kernel(const HeadArgs a) {
  __shared__ uint32_t part[kWavesPerBlock], mine, out;
  __shared__ float most[kWavesPerBlock];
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
  int64_t target[4];
  float w[4], top = 0.0f;
  uint32_t has = 0;
  if (t == 0) mine = 0xFFFFFFFFu;
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j) {
    const uint32_t r = 4 * t + j;
    target[j] = r < a.rows ? a.targets[r] : -1;
    w[j] = r < a.rows && a.row_weight ? a.row_weight[r] : 1.0f;
    if (target[j] >= 0 && target[j] < (int64_t)a.vocab) {
      has |= 1u << j;
      if (fabsf(w[j]) < INFINITY) top = fmaxf(top, fabsf(w[j]));
    }
  }
  uint32_t sum = __popc(has);
#pragma unroll
  for (uint32_t s = 1; s < 64; s <<= 1) {
    const uint32_t up = __shfl_up(sum, s, 64);
    if (lane >= s) sum += up;
    top = fmaxf(top, __shfl_xor(top, (int)s, 64));
  }
  if (lane == 63) part[wave] = sum;
  if (lane == 0) most[wave] = top;
  __syncthreads();
  uint32_t live = 0, at = sum - __popc(has);
#pragma unroll
  for (uint32_t i = 0; i < kWavesPerBlock; ++i) {
    at += i < wave ? part[i] : 0;
    live += part[i];
    top = fmaxf(top, most[i]);
  }
  if (t == blockIdx.x / 4) out = !(has >> (blockIdx.x % 4) & 1);
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j) {
    const uint32_t r = 4 * t + j;
    const bool counts = has >> j & 1;
    if (counts && at == blockIdx.x) mine = r;
    if (blockIdx.x == 0 && r < a.rows) {
      a.counts[r] = counts;
      if (counts) {
        a.row_of[at] = r;
        a.target[at] = (uint32_t)target[j];
        const float omega = top > 0.0f ? w[j] / top : w[j];
        a.omega[at] = omega;
        if (a.lift) a.lift[at] = lift_of(omega);
      } else {
        a.logp[r] = 0.0f;
        a.terms[r] = 0.0;
      }
    }
    at += counts;
  }
  if (blockIdx.x == 0 && t == 0)
    *a.meta = Meta{live, (float)(a.coef * (double)top / kHeld), splits_for(a, live)};
  __syncthreads();
  gather_row(a, live, blockIdx.x, mine, a.dhidden && out);
}

// Block i: the i-th row that counts is copied; row i's gradient, if it does not
// count, is zero.
__global__ void __launch_bounds__(kBlock) gather_kernel(const HeadArgs a) {
  for (uint32_t i = blockIdx.x; i < a.rows; i += gridDim.x)
    gather_row(a, a.meta->live, i, i < a.meta->live ? a.row_of[i] : 0xFFFFFFFFu, a.dhidden && !a.counts[i]);
}

// Tile numbers in an order that keeps a group of tiles on one XCD: each XCD
// takes a contiguous run, in which eight m tiles go along n together.
__device__ __forceinline__ void tile_of(uint32_t b, uint32_t mt, uint32_t nt, uint32_t* m, uint32_t* n) {
  const uint32_t i = (uint32_t)xcd_contiguous(b, (uint64_t)mt * nt);
  constexpr uint32_t G = 8;
  const uint32_t group = i / (G * nt), in = i % (G * nt), size = min(G, mt - group * G);
  *m = group * G + in % size;
  *n = in / size;
}

// ---------------------------------------------------------------------------
// Product one.  PLANES of the exponentials are kept, in fp16.
// ---------------------------------------------------------------------------
template <int DT, class T, int PLANES>
__global__ void __launch_bounds__(kGemmThreads, 2) logits_kernel(const HeadArgs a) {
  extern __shared__ __align__(16) char lds[];
  const uint32_t live = a.meta->live, mt = (live + T::kM - 1) / T::kM;
  if (blockIdx.x >= mt * a.tiles) return;
  uint32_t tm, tn;
  tile_of(blockIdx.x, mt, a.tiles, &tm, &tn);
  Rows<T::kM> p;
  Rows<256> q;
  p.begin(a.kept, (uint64_t)tm * T::kM, live, a.dim, a.dim);
  q.begin(a.weight, (uint64_t)tn * 256, a.vocab, a.weight_stride, a.dim);
  typename T::Acc acc;
  clear<T>(acc);
  gemm_tile<DT, T>(p, q, 0, a.dim, (lds_char*)lds, acc);
  // the tile's maximum of each row, over the wavefronts that share it
  constexpr int W = T::kWavesN;
  const uint32_t t = thread_anew(), lane = t & 63, share = wave_of_block() % W * T::kM;
  float* red = reinterpret_cast<float*>(lds + T::kM * 512);  // behind the tile's exponentials in 16 bits
  const auto most = [&](uint32_t r) {
    float m = red[r];
#pragma unroll
    for (int w = 1; w < W; ++w) m = fmaxf(m, red[w * T::kM + r]);
    return m;
  };
  __syncthreads();
#pragma unroll
  for (int i = 0; i < T::kI; ++i) {
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < T::kJ; ++j)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (tn * 256 + T::column(j, t) + x < a.vocab) top = fmaxf(top, acc[i][j][x]);
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    if (lane < 16) red[share + T::row(i, t)] = top;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < T::kI; ++i) {
    const uint32_t r = T::row(i, t), row = tm * T::kM + r;
    const bool has = row < live;
    const float top = most(r), m = top == -INFINITY ? 0.0f : top;
    const uint32_t target = has ? a.target[row] : 0xFFFFFFFFu;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < T::kJ; ++j) {
      const uint32_t n0 = tn * 256 + T::column(j, t);
      float e[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint32_t n = n0 + x;
        e[x] = n < a.vocab ? __builtin_amdgcn_exp2f((acc[i][j][x] - m) * a.c) : 0.0f;
        if (n == target) a.said[row] = acc[i][j][x];
        else sum += e[x];
      }
      if constexpr (PLANES > 0) put_quad<ZERO_F16>(lds, r, T::column(j, t), f32x4{e[0], e[1], e[2], e[3]} * kTileExp);
    }
    sum += __shfl_xor(sum, 16, 64);
    sum += __shfl_xor(sum, 32, 64);
    if (lane < 16) red[W * T::kM + share + r] = sum;
  }
  __syncthreads();
  if (t < T::kM && tm * T::kM + t < live) {
    const uint32_t r = t;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) sum += red[(W + w) * T::kM + r];
    a.stats[(uint64_t)(tm * T::kM + r) * a.tiles + tn] = f32x2{most(r), sum};
  }
  if constexpr (PLANES > 0)
    store_rows<T::kM>(lds, 256, t, [&](uint32_t m) {
      const uint32_t row = tm * T::kM + m;
      return row < live ? a.held + (uint64_t)row * a.padded + tn * 256 : nullptr;
    });
  if constexpr (PLANES > 1) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < T::kI; ++i) {
      const uint32_t r = T::row(i, t);
      const float top = most(r), m = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int j = 0; j < T::kJ; ++j) {
        f32x4 rest;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float e = tn * 256 + T::column(j, t) + x < a.vocab ? __builtin_amdgcn_exp2f((acc[i][j][x] - m) * a.c) * kTileExp : 0.0f;
          rest[x] = e - rounded<ZERO_F16>(e);
        }
        put_quad<ZERO_F16>(lds, r, T::column(j, t), rest);
      }
    }
    __syncthreads();
    store_rows<T::kM>(lds, 256, t, [&](uint32_t m) {
      const uint32_t row = tm * T::kM + m;
      return row < live ? a.held + ((uint64_t)live + row) * a.padded + tn * 256 : nullptr;
    });
  }
}

// LDS of that: the products' slots, then the exponentials and two numbers of each row and wavefront.
template <class T>
constexpr uint32_t logits_lds() {
  constexpr uint32_t after = T::kM * 512 + 2 * T::kWavesN * T::kM * 4;
  return after > (uint32_t)T::kLds ? after : T::kLds;
}

// The same for up to kFewRows rows, bound by the reading of the weights: a wavefront
// reads the weights of 16 columns straight into registers, 16 bytes to a lane,
// kFewSteps steps of 32 k in flight; the rows' hidden states come from the
// caches.  The four wavefronts of a block take turns along k.  (One row of 32,000 x
// 4096 bf16 64 us with it, 77 with the products' tiles; 16 rows 79 and 78: the
// hidden states, read by every wavefront, then cost as much as the barriers saved.)
constexpr uint32_t kFewRows = 8, kFewShift = 4;
constexpr int kFewSteps = 4;

template <int DT, int PLANES>
__global__ void __launch_bounds__(kBlock) few_logits_kernel(const HeadArgs a) {
  __shared__ f32x4 share[kWavesPerBlock - 1][64];
  const uint32_t live = a.meta->live, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (live == 0) return;
  const uint32_t tn = blockIdx.x, column = tn * 16, row = lane % 16, k0 = lane / 16 * 8;
  const bool has = row < live, in = column + lane % 16 < a.vocab;
  const uint16_t* w = static_cast<const uint16_t*>(a.weight) + (uint64_t)(in ? column + lane % 16 : 0) * a.weight_stride + k0;
  const uint16_t* h = a.kept + (uint64_t)(has ? row : 0) * a.dim + k0;
  f32x4 acc = {0, 0, 0, 0};
  for (uint32_t k = wave * 32 * kFewSteps; k < a.dim; k += kWavesPerBlock * 32 * kFewSteps) {
    u32x4 x[kFewSteps], y[kFewSteps];
    if (k + 32 * kFewSteps <= a.dim) {
#pragma unroll
      for (int i = 0; i < kFewSteps; ++i) x[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w + k + 32 * i));
#pragma unroll
      for (int i = 0; i < kFewSteps; ++i) y[i] = has ? *reinterpret_cast<const u32x4*>(h + k + 32 * i) : u32x4{0, 0, 0, 0};
    } else {
#pragma unroll
      for (int i = 0; i < kFewSteps; ++i) {
        const bool on = k + k0 + 32 * i < a.dim;
        x[i] = on ? *reinterpret_cast<const u32x4*>(w + k + 32 * i) : u32x4{0, 0, 0, 0};
        y[i] = on && has ? *reinterpret_cast<const u32x4*>(h + k + 32 * i) : u32x4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int i = 0; i < kFewSteps; ++i) acc = mfma16<DT>(x[i], y[i], acc);
  }
  if (wave > 0) share[wave - 1][lane] = acc;
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int i = 0; i < kWavesPerBlock - 1; ++i) acc += share[i][lane];
  // acc[x]: column + 4 (lane / 16) + x of row lane % 16
  const uint32_t n0 = column + lane / 16 * 4;
  float top = -INFINITY;
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (n0 + x < a.vocab) top = fmaxf(top, acc[x]);
  top = fmaxf(top, __shfl_xor(top, 16, 64));
  top = fmaxf(top, __shfl_xor(top, 32, 64));
  const float m = top == -INFINITY ? 0.0f : top;
  const uint32_t target = has ? a.target[row] : 0xFFFFFFFFu;
  float sum = 0.0f, e[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    e[x] = n0 + x < a.vocab ? __builtin_amdgcn_exp2f((acc[x] - m) * a.c) : 0.0f;
    if (n0 + x == target) a.said[row] = acc[x];
    else sum += e[x];
  }
  if (PLANES > 0 && has) {
#pragma unroll
    for (int p = 0; p < PLANES; ++p) {
      float y[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) y[x] = p == 0 ? e[x] * kTileExp : e[x] * kTileExp - rounded<ZERO_F16>(e[x] * kTileExp);
      store4<ZERO_F16>(a.held, ((uint64_t)p * live + row) * a.padded + n0, y[0], y[1], y[2], y[3]);
    }
  }
  sum += __shfl_xor(sum, 16, 64);
  sum += __shfl_xor(sum, 32, 64);
  // the blocks behind the vocabulary only store zeros
  if (lane < live && lane < 16 && tn < a.tiles) a.stats[(uint64_t)lane * a.tiles + tn] = f32x2{top, sum};
}

// ---------------------------------------------------------------------------
// Log-probabilities, and dx in place of the exponentials.  Blocks (row, part of
// the row): each goes over the row's tile statistics and then its own part.
// ---------------------------------------------------------------------------
constexpr uint32_t kPartTiles = 512;      // most tiles of one part

template <int DT, int PLANES>
__global__ void __launch_bounds__(kBlock) softmax_kernel(const HeadArgs a) {
  __shared__ float scale[PLANES > 0 ? kPartTiles : 1];
  __shared__ double part[kWavesPerBlock];
  __shared__ float tops[kWavesPerBlock];
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6, live = a.meta->live;
  // this block's tiles
  const uint32_t per = (a.tiles + gridDim.y - 1) / gridDim.y, tile0 = blockIdx.y * per, tile1 = min(tile0 + per, a.tiles);
  for (uint32_t row = blockIdx.x; row < live; row += gridDim.x) {
    const f32x2* stats = a.stats + (uint64_t)row * a.tiles;
    float top = -INFINITY;
    for (uint32_t i = t; i < a.tiles; i += kBlock) top = fmaxf(top, stats[i][0]);
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) top = fmaxf(top, __shfl_xor(top, s, 64));
    __syncthreads();
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    for (int i = 0; i < kWavesPerBlock; ++i) top = fmaxf(top, tops[i]);
    double sum = 0.0;
    for (uint32_t i = t; i < a.tiles; i += kBlock) {
      const f32x2 s = stats[i];
      if (!(s[1] == 0.0f && s[0] == -INFINITY)) sum += (double)s[1] * (double)__builtin_amdgcn_exp2f((s[0] - top) * a.c);
    }
    sum = row_sum<kWavesPerBlock>(sum, part);
    const uint32_t target = a.target[row], from = a.row_of[row];
    const double d = (double)(a.said[row] - top) * a.inv_temperature;
    const double all = sum + exp(d);
    if (t == 0 && blockIdx.y == 0) {
      const double lp = d == 0.0 ? -log1p(sum) : d - log(all);
      a.logp[from] = (float)lp;
      a.terms[from] = lp * (a.row_weight ? (double)a.row_weight[from] : 1.0);
    }
    if constexpr (PLANES > 0) {
      // lifted, and lowered at once where no product reads it so
      const float lift = DT == ZERO_F16 && a.lift ? a.lift[row] : 1.0f;
      const float omega = a.omega[row] * kHeld * lift;
      const float unit = (float)((double)omega / all) * (1.0f / kTileExp);
      float other = -(float)((double)omega * (sum / all));  // at the target: p - 1, without cancellation
      const bool lower = DT == ZERO_F16 && lift != 1.0f && !a.dhidden;
      const float down = inverse_of(lift);
      if (lower) other *= down;
      if (t == 0 && blockIdx.y == 0) {
        const float rest = other - in_planes<DT>(other, PLANES);
        a.rest[row] = rest;
        if (a.low != a.rest) a.low[row] = rest;
      }
      uint16_t* const held = a.held + (uint64_t)row * a.padded;
      uint16_t* const second = a.held + ((uint64_t)live + row) * a.padded;  // of two
      for (uint32_t first = tile0; first < tile1; first += kPartTiles) {
        const uint32_t end = min(first + kPartTiles, tile1);
        __syncthreads();
        for (uint32_t i = t; i < end - first; i += kBlock) {
          const float m = stats[first + i][0];
          scale[i] = m == -INFINITY ? 0.0f : unit * __builtin_amdgcn_exp2f((m - top) * a.c);
        }
        __syncthreads();
        const uint32_t v0 = (first << a.shift) / 8, v1 = min(end << a.shift, a.padded) / 8;
#pragma unroll 4
        for (uint32_t v = v0 + t; v < v1; v += kBlock) {
          const Vec<ZERO_F16>::Raw e = load8<ZERO_F16>(held, (uint64_t)v * 8);
          Vec<ZERO_F16>::Raw e2 = e;
          if constexpr (PLANES > 1) e2 = load8<ZERO_F16>(second, (uint64_t)v * 8);
          const float f = scale[(v - v0) >> (a.shift - 3)];
          float x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float y = Vec<ZERO_F16>::get(e, k);
            if constexpr (PLANES > 1) y += Vec<ZERO_F16>::get(e2, k);
            y *= f;
            if (lower) y = in_planes<DT>(y, PLANES) * down;  // the roundings of a row that is lowered later
            x[k] = v * 8 + k == target ? other : y;
          }
          store8<DT>(held, (uint64_t)v * 8, x);
          if constexpr (PLANES > 1) {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] -= rounded<DT>(x[k]);
            store8<DT>(second, (uint64_t)v * 8, x);
          }
        }
      }
    }
  }
}

// (A launch of its own also for few rows: as the last block's work in softmax_kernel, behind
// a counter and its fences, the sum made scores of 1 to 128 rows no faster, alone
// or among others, and 77 rows of 50,001 x 1000 fp16 with gradients 161 us alone
// instead of 154.)
__global__ void __launch_bounds__(kBlock) loss_kernel(const double* terms, const uint8_t* counts, uint64_t n, double inv_divisor,
                                                      float* stats) {
  __shared__ double part[kWavesPerBlock];
  double sum = 0.0, count = 0.0;
  for (uint64_t i = threadIdx.x; i < n; i += kBlock) {
    sum += terms[i];
    count += (double)counts[i];
  }
  sum = row_sum<kWavesPerBlock>(sum, part);
  count = row_sum<kWavesPerBlock>(count, part);
  if (threadIdx.x == 0) {
    stats[0] = (float)(-sum * inv_divisor);
    stats[1] = (float)count;
  }
}

// ---------------------------------------------------------------------------
// Products two and three.
// ---------------------------------------------------------------------------
template <int DT, class T>
__global__ void __launch_bounds__(kGemmThreads, 2) dhidden_kernel(const HeadArgs a) {
  extern __shared__ __align__(16) char lds[];
  const uint32_t live = a.planes * a.meta->live, splits = a.meta->splits;  // rows of dx
  const uint32_t mt = (live + T::kM - 1) / T::kM, nt = (a.dim + 255) / 256;
  const bool whole = splits == 1 && a.planes == 1;
  if (live == 0) return;
  const uint32_t steps = (a.vocab + 63) / 64, per = (steps + splits - 1) / splits;
  const uint32_t split = blockIdx.x / (mt * nt);
  if (split >= splits) return;
  uint32_t tm, tn;
  tile_of(blockIdx.x % (mt * nt), mt, nt, &tm, &tn);
  const uint32_t k_end = min((split + 1) * per * 64, a.vocab);
  Rows<T::kM> p;
  Columns<256> q;
  // the columns behind the vocabulary hold zeros
  p.begin(a.held, (uint64_t)tm * T::kM, live, a.padded, (k_end + 7) / 8 * 8);
  q.begin(a.weight, (uint64_t)tn * 256, a.dim, a.weight_stride, k_end);
  typename T::Acc acc;
  clear<T>(acc);
  gemm_tile<DT, T>(p, q, split * per * 64, k_end, (lds_char*)lds, acc);
  const uint32_t t = thread_anew();
  if (whole) {  // what the targets' entries lost
#pragma unroll
    for (int i = 0; i < T::kI; ++i) {
      const uint32_t row = tm * T::kM + T::row(i, t);
      if (row >= live) continue;
      const float rest = a.rest[row];
      const uint16_t* w = static_cast<const uint16_t*>(a.weight) + a.target[row] * a.weight_stride;
#pragma unroll
      for (int j = 0; j < T::kJ; ++j) {
        const uint32_t n = tn * 256 + T::column(j, t);
        if (n >= a.dim) continue;
        const u32x2 v = *reinterpret_cast<const u32x2*>(w + n);
        const typename Vec<DT>::Raw r = {u32x4{v[0], v[1], 0, 0}};
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[i][j][x] = fmaf(rest, Vec<DT>::get(r, x), acc[i][j][x]);
        if constexpr (DT == ZERO_F16) {
          if (a.lift) acc[i][j] *= inverse_of(a.lift[row]);
        }
      }
    }
  }
  if (whole) {
    __syncthreads();
    uint16_t* out = static_cast<uint16_t*>(a.dhidden) + tn * 256;
    store_tile<DT, T>(acc, a.meta->factor, a.dim - tn * 256, lds, t, [&](uint32_t m) {
      const uint32_t row = tm * T::kM + m;
      return row < live ? out + a.row_of[row] * a.dhidden_stride : nullptr;
    });
    return;
  }
#pragma unroll
  for (int i = 0; i < T::kI; ++i) {
    const uint32_t row = tm * T::kM + T::row(i, t);
    if (row >= live) continue;
#pragma unroll
    for (int j = 0; j < T::kJ; ++j) {
      const uint32_t n = tn * 256 + T::column(j, t);
      if (n < a.dim) *reinterpret_cast<f32x4*>(a.part + ((uint64_t)split * live + row) * a.dim + n) = acc[i][j];
    }
  }
}

// dhidden from the sums over parts of the vocabulary and of dx's numbers, in their
// order, and what the target's entry lost.  Lifted rows of dx are lowered for dweight's product.
template <int DT>
__global__ void __launch_bounds__(kBlock) join_kernel(const HeadArgs a) {
  const uint32_t live = a.meta->live, parts = a.meta->splits * a.planes;
  const bool lower = DT == ZERO_F16 && a.lift && a.dweight;
  if (parts <= 1 && !lower) return;
  const float f = a.meta->factor;
  for (uint32_t row = blockIdx.x; row < live; row += gridDim.x) {
    const float rest = a.rest[row], lift = DT == ZERO_F16 && a.lift ? a.lift[row] : 1.0f, down = inverse_of(lift);
    const uint32_t target = a.target[row];
    if (parts > 1) {
      const uint64_t at = a.row_of[row] * a.dhidden_stride;
      const u32x2* w = reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(a.weight) + target * a.weight_stride);
      for (uint32_t v = blockIdx.y * kBlock + threadIdx.x; v < a.dim / 4; v += gridDim.y * kBlock) {
        f32x4 x = {0, 0, 0, 0};
#pragma unroll 8
        for (uint32_t s = 0; s < parts; ++s)
          x += *reinterpret_cast<const f32x4*>(a.part + ((uint64_t)s * live + row) * a.dim + v * 4);
        const typename Vec<DT>::Raw r = {u32x4{w[v][0], w[v][1], 0, 0}};
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = fmaf(rest, Vec<DT>::get(r, k), x[k]);
        if constexpr (DT == ZERO_F16) x *= down;
        x *= f;
        store4<DT>(a.dhidden, at + v * 4, x[0], x[1], x[2], x[3]);
      }
    }
    if constexpr (DT == ZERO_F16) {
      if (!lower || lift == 1.0f) continue;
      uint16_t* const held = a.held + (uint64_t)row * a.padded;
      uint16_t* const second = a.held + ((uint64_t)live + row) * a.padded;
      for (uint32_t v = blockIdx.y * kBlock + threadIdx.x; v < a.padded / 8; v += gridDim.y * kBlock) {
        const typename Vec<DT>::Raw e = load8<DT>(held, (uint64_t)v * 8);
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = Vec<DT>::get(e, k);
        if (a.planes > 1) {
          const typename Vec<DT>::Raw e2 = load8<DT>(second, (uint64_t)v * 8);
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] += Vec<DT>::get(e2, k);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (v * 8 + k == target) x[k] += rest;  // what the entry was
          x[k] *= down;
          if (v * 8 + k == target) a.low[row] = x[k] - in_planes<DT>(x[k], a.planes);
        }
        store8<DT>(held, (uint64_t)v * 8, x);
        if (a.planes > 1) {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] -= rounded<DT>(x[k]);
          store8<DT>(second, (uint64_t)v * 8, x);
        }
      }
    }
  }
}

// What the targets' entries lost, as terms of dweight's product: of the rows whose
// target lies in the tile, in their order and 64 at a time, P holds the residual at
// the target's column (zeros elsewhere) and Q the row's hidden state.
template <int DT, class T>
__device__ __forceinline__ void add_rests(const HeadArgs& a, uint32_t live, uint32_t tm, uint32_t tn, char* lds,
                                          uint32_t t, typename T::Acc& acc) {
  typedef Columns<T::kM> P;
  typedef Columns<256> Q;
  constexpr uint32_t kList = 4096, kEach = 4;  // consecutive rows to a thread
  static_assert(T::kBytesP == 64 * 2 * T::kM, "half of the bytes of P are 32 rows");
  static_assert(T::kSlotBytes + kList * 4 + 2 * kWaves * 4 <= T::kLds, "the list lies in the second slot");
  uint32_t* list = reinterpret_cast<uint32_t*>(lds + T::kSlotBytes);  // rows, the i-th at i % kList
  uint32_t* parts = list + kList;  // the wavefronts' counts, in turn
  const uint32_t lane = t & 63, wave = wave_of_block();
  const uint32_t m0 = wave / T::kWavesN * T::kWaveM, n0 = wave % T::kWavesN * T::kWaveN;
  uint32_t found = 0, used = 0, turn = 0, next[kEach];
#pragma unroll
  for (uint32_t i = 0; i < kEach; ++i) next[i] = kEach * t + i < live ? a.target[kEach * t + i] : 0xFFFFFFFFu;
  for (uint32_t r0 = 0; r0 < live; r0 += kEach * kGemmThreads, turn ^= kWaves) {
    const uint32_t r = r0 + kEach * t, ahead = r + kEach * kGemmThreads;
    uint32_t target[kEach];
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) {
      target[i] = next[i];
      next[i] = ahead + i < live ? a.target[ahead + i] : 0xFFFFFFFFu;
    }
    uint32_t mine = 0, before = 0, all = 0;
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) {
      const bool hit = target[i] != 0xFFFFFFFFu && target[i] - tm * T::kM < (uint32_t)T::kM;
      const uint64_t hits = __ballot(hit);
      mine |= (uint32_t)hit << i;
      before += (uint32_t)__popcll(hits & ((1ull << lane) - 1));
      all += (uint32_t)__popcll(hits);
    }
    const bool last = r0 + kEach * kGemmThreads >= live;
    uint32_t* part = parts + turn;
    if (lane == 0) part[wave] = all;
    __syncthreads();
    uint32_t at = found + before;
    for (uint32_t w = 0; w < kWaves; ++w) {
      at += w < wave ? part[w] : 0;
      found += part[w];
    }
    if (found == used) continue;
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i)
      if (mine >> i & 1) list[at++ % kList] = r + i;
    while (found - used >= 64 || (last && found > used)) {
      const uint32_t n = min(found - used, 64u), halves = (n + 31) / 32;
      // zeros, and the hidden states
      for (uint32_t i = t; i < T::kBytesP / 32 * halves; i += kGemmThreads)
        *reinterpret_cast<u32x4*>(lds + i * 16) = u32x4{0, 0, 0, 0};
      __syncthreads();
#pragma unroll 2
      for (uint32_t i = t; i < halves * 32 * 32; i += kGemmThreads) {
        const uint32_t k = i / 32, c = i % 32, column = tn * 256 + c * 8;
        u32x4 v = {0, 0, 0, 0};
        if (k < n && column < a.dim) v = *reinterpret_cast<const u32x4*>(a.kept + (uint64_t)list[(used + k) % kList] * a.dim + column);
        *reinterpret_cast<u32x4*>(lds + T::kBytesP + k * 512 + (c ^ Q::swizzle(k)) * 16) = v;
      }
      if (t < n) {
        const uint32_t k = t, row = list[(used + k) % kList], m = a.target[row] - tm * T::kM;
        *reinterpret_cast<uint16_t*>(lds + k * (2 * T::kM) + ((m / 8) ^ P::swizzle(k)) * 16 + m % 8 * 2) =
            (uint16_t)Vec<DT>::pack(a.low[row], 0.0f);
      }
      __syncthreads();
#pragma unroll 1
      for (uint32_t kk = 0; kk < halves; ++kk) {
        u32x4 q[T::kJ];
#pragma unroll
        for (int j = 0; j < T::kJ; ++j) q[j] = Q::fragment((lds_char*)lds + T::kBytesP, n0 + 16 * j, kk, lane);
#pragma unroll
        for (int i = 0; i < T::kI; ++i) {
          const u32x4 p = P::fragment((lds_char*)lds, m0 + 16 * i, kk, lane);
#pragma unroll
          for (int j = 0; j < T::kJ; ++j) acc[i][j] = mfma16<DT>(q[j], p, acc[i][j]);
          __builtin_amdgcn_sched_barrier(0);  // few registers are left beside the sums
        }
      }
      __syncthreads();
      used += n;
    }
  }
}

template <int DT, class T>
__global__ void __launch_bounds__(kGemmThreads, 2) dweight_kernel(const HeadArgs a) {
  extern __shared__ __align__(16) char lds[];
  const uint32_t live = a.meta->live, mt = (a.vocab + T::kM - 1) / T::kM, nt = (a.dim + 255) / 256;
  uint32_t tm, tn;
  tile_of(blockIdx.x, mt, nt, &tm, &tn);
  typename T::Acc acc;
  clear<T>(acc);
  add_rests<DT, T>(a, live, tm, tn, lds, thread_anew(), acc);
  Columns<T::kM> p;
  Columns<256> q;
  const uint32_t rows = a.planes * live;  // of dx
  p.begin(a.held, (uint64_t)tm * T::kM, a.padded, a.padded, rows);
  q.begin(a.kept, (uint64_t)tn * 256, a.dim, a.dim, rows);
  gemm_tile<DT, T>(p, q, 0, rows, (lds_char*)lds, acc);
  const uint32_t t = thread_anew();
  const float f = a.meta->factor;
  if (a.first && a.last) {
    __syncthreads();
    uint16_t* out = static_cast<uint16_t*>(a.dweight) + tn * 256;
    store_tile<DT, T>(acc, f, a.dim - tn * 256, lds, t, [&](uint32_t m) {
      const uint32_t row = tm * T::kM + m;
      return row < a.vocab ? out + row * a.dweight_stride : nullptr;
    });
    return;
  }
#pragma unroll
  for (int i = 0; i < T::kI; ++i) {
    const uint32_t row = tm * T::kM + T::row(i, t);
    if (row >= a.vocab) continue;
#pragma unroll
    for (int j = 0; j < T::kJ; ++j) {
      const uint32_t n = tn * 256 + T::column(j, t);
      if (n >= a.dim) continue;
      f32x4 x = acc[i][j] * f;
      f32x4* sum = reinterpret_cast<f32x4*>(a.sum + (uint64_t)row * a.dim + n);
      if (!a.first) x += *sum;
      if (a.last) store4<DT>(a.dweight, row * a.dweight_stride + n, x[0], x[1], x[2], x[3]);
      else *sum = x;
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
constexpr uint32_t kMaxDim = 1u << 15;

struct Space {
  uint64_t meta, row_of, target, omega, said, rest, lift, low, terms, counts, kept, held, stats, part, sum, bytes;
  uint32_t piece, tiles, shift;
};

// Where the pieces of `piece_rows` rows have their intermediates.
Space space_of(uint64_t n_rows, uint32_t vocab, uint32_t dim, uint32_t piece_rows, bool grad) {
  Space s = {};
  s.piece = (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(n_rows, piece_rows));
  static_assert(kFewShift == 4, "the statistics below are of 16-column tiles");
  s.shift = s.piece <= kFewRows ? kFewShift : 8;
  s.tiles = (vocab + (1u << s.shift) - 1) >> s.shift;
  const uint64_t p = s.piece, padded = (vocab + 255) / 256 * 256;
  // rows of dx, the most of any number of rows up to p
  const uint64_t few = std::min<uint64_t>(p, kTwoRows), held = grad ? std::max(planes_of(s.piece, dim) * p, 2 * few) : p;
  uint64_t at = 0;
  const auto take = [&](uint64_t bytes) {
    const uint64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  s.meta = take(sizeof(Meta));
  s.row_of = take(p * 4);
  s.target = take(p * 4);
  s.omega = take(p * 4);
  s.said = take(p * 4);
  s.rest = take(grad ? p * 4 : 0);
  s.lift = take(grad ? p * 4 : 0);
  s.low = take(grad ? p * 4 : 0);
  s.terms = take(n_rows * 8);
  s.counts = take(n_rows);
  s.kept = take(held * dim * 2);
  // the most of any number of rows up to p: a workspace serves fewer rows too
  s.stats = take(std::max(p * ((vocab + 255) / 256), std::min<uint64_t>(p, kFewRows) * ((vocab + 15) / 16)) * 8);
  s.held = take(grad ? held * padded * 2 : 0);
  uint64_t part = 0;  // dhidden's parts, for whatever number of rows counts
  for (uint64_t most : {(uint64_t)128, held}) {  // the last piece may be smaller, and so may a later call
    const uint64_t rows = std::min(most, held);
    const uint32_t t = tile_rows((uint32_t)rows);
    for (uint32_t m = t; grad && m < rows + t; m += t) {
      const uint32_t n = splits_of(m / t, vocab, dim);
      if (n > 1 || m <= 2 * kTwoRows || dim <= kTwoDim) part = std::max(part, n * std::min<uint64_t>(m, rows));
    }
  }
  s.part = take(part * dim * 4);
  s.sum = take(grad && n_rows > p ? (uint64_t)vocab * dim * 4 : 0);
  s.bytes = at;
  return s;
}

int check_shape(uint64_t n_rows, uint32_t vocab, uint32_t dim, uint32_t piece_rows, const char* who) {
  if (vocab == 0 || vocab > 1u << 20) return fail(ZERO_EINVAL, "%s: vocab %u outside [1, 2^20]", who, vocab);
  if (dim == 0 || dim > kMaxDim || dim % 8)
    return fail(ZERO_EINVAL, "%s: dim %u is not a multiple of 8 in [8, %u]", who, dim, kMaxDim);
  if (piece_rows == 0 || piece_rows > 16384) return fail(ZERO_EINVAL, "%s: piece_rows %u outside [1, 16384]", who, piece_rows);
  if (n_rows > (uint64_t)INT32_MAX) return fail(ZERO_EINVAL, "%s: n_rows beyond 2^31 - 1", who);
  return ZERO_OK;
}

int check_matrix(const void* p, uint32_t dim, uint64_t stride, const char* name, const char* who) {
  if (!p || !multiple_of(p, 16) || stride % 8)
    return fail(ZERO_EINVAL, "%s: %s is NULL, or its rows are not 16-byte aligned", who, name);
  if (stride < dim || stride > (1u << 22))
    return fail(ZERO_EINVAL, "%s: %s has a row stride of %llu outside [dim, 2^22]", who, name, (unsigned long long)stride);
  return ZERO_OK;
}

// Calls fn with the tile of a piece's rows.
template <typename F>
void by_tile(uint32_t rows, F fn) {
  if (tile_rows(rows) == 128) fn(Middle{});
  else fn(Wide{});
}

template <int DT, int PLANES>
void launch_rows(const HeadArgs& a, hipStream_t stream) {
  if (a.shift == kFewShift) {
    hipLaunchKernelGGL((few_logits_kernel<DT, PLANES>), a.padded >> kFewShift, kBlock, 0, stream, a);
  } else {
    by_tile(a.rows, [&](auto tile) {
      typedef decltype(tile) T;
      hipLaunchKernelGGL((logits_kernel<DT, T, PLANES>), (a.rows + T::kM - 1) / T::kM * a.tiles, kGemmThreads, logits_lds<T>(),
                         stream, a);
    });
  }
  // with few rows, parts of them: 1024 blocks, of 2048 columns at least
  const uint32_t parts = PLANES > 0 ? std::min((a.padded + 2047) / 2048, std::max(1024 / a.rows, 1u)) : 1;
  hipLaunchKernelGGL((softmax_kernel<DT, PLANES>), dim3(a.rows, parts), kBlock, 0, stream, a);
}

template <int DT>
void launch_dweight(const HeadArgs& a, hipStream_t stream) {
  const uint32_t tiles = (a.vocab + 255) / 256 * ((a.dim + 255) / 256);
  hipLaunchKernelGGL((dweight_kernel<DT, Wide>), tiles, kGemmThreads, Wide::kLds, stream, a);
}

template <int DT>
void launch_piece(HeadArgs a, bool grad, hipStream_t stream) {
  const uint32_t nt = (a.dim + 255) / 256, rows = a.planes * a.rows;
  uint32_t blocks = 0;  // the most that dhidden's product has, whatever number of rows counts
  for (uint32_t i = 0; grad && i * tile_rows(rows) < rows; ++i) {
    a.splits[i] = (uint8_t)splits_of(i + 1, a.vocab, a.dim);
    blocks = std::max(blocks, (i + 1) * nt * a.splits[i]);
  }
  if (a.rows <= kGatherRows) {
    hipLaunchKernelGGL(prepare_few_kernel, a.rows, kBlock, 0, stream, a);
  } else {
    hipLaunchKernelGGL(prepare_kernel, 1, 1024, 0, stream, a);
    hipLaunchKernelGGL(gather_kernel, a.rows, kBlock, 0, stream, a);
  }
  if (!grad) return launch_rows<DT, 0>(a, stream);
  if (a.planes == 2) launch_rows<DT, 2>(a, stream);
  else launch_rows<DT, 1>(a, stream);
  if (a.dhidden) {
    by_tile(rows, [&](auto tile) {
      typedef decltype(tile) T;
      hipLaunchKernelGGL((dhidden_kernel<DT, T>), blocks, kGemmThreads, T::kLds, stream, a);
    });
    uint32_t parts = (a.dim / 4 + kBlock - 1) / kBlock;
    if (a.lift && a.dweight)  // which rows are lowered is not known here: with few, parts of them
      parts = std::max(parts, std::min((a.padded / 8 + 4 * kBlock - 1) / (4 * kBlock), 2048 / a.rows));
    hipLaunchKernelGGL(join_kernel<DT>, dim3(a.rows, parts), kBlock, 0, stream, a);
  }
  if (a.dweight) launch_dweight<DT>(a, stream);
}

}  // namespace
}  // namespace zs

using namespace zs;

extern "C" int zero_linear_cross_entropy_workspace_bytes(uint64_t n_rows, uint32_t vocab, uint32_t dim, uint32_t piece_rows,
                                                         int grad, uint64_t* bytes) {
  static const char* who = "zero_linear_cross_entropy_workspace_bytes";
  clear_error();
  if (!bytes) return fail(ZERO_EINVAL, "%s: bytes is NULL", who);
  const int rc = check_shape(n_rows, vocab, dim, piece_rows, who);
  if (rc) return rc;
  *bytes = space_of(n_rows, vocab, dim, piece_rows, grad != 0).bytes;
  return ZERO_OK;
}

extern "C" int zero_linear_cross_entropy(const zero_linear_cross_entropy_args* p, hipStream_t stream) {
  static const char* who = "zero_linear_cross_entropy";
  clear_error();
  if (!p) return fail(ZERO_EINVAL, "%s: args is NULL", who);
  if (p->dtype != ZERO_F16 && p->dtype != ZERO_BF16) return fail(ZERO_EINVAL, "%s: dtype %d is not fp16 or bf16", who, p->dtype);
  int rc = check_shape(p->n_rows, p->vocab, p->dim, p->piece_rows, who);
  if (rc) return rc;
  const double nums[] = {p->divisor, p->temperature, p->grad_scale};
  for (double x : nums)
    if (!std::isfinite(x)) return fail(ZERO_EINVAL, "%s: non-finite parameter", who);
  if (p->divisor <= 0.0) return fail(ZERO_EINVAL, "%s: divisor must be > 0", who);
  if (p->temperature <= 0.0 || !std::isnormal((float)(kLog2e / p->temperature)))
    return fail(ZERO_EINVAL, "%s: temperature %g is out of range", who, p->temperature);
  if (!p->stats || !multiple_of(p->stats, 4)) return fail(ZERO_EINVAL, "%s: stats is NULL or misaligned", who);
  if ((rc = check_matrix(p->weight, p->dim, p->weight_stride, "weight", who))) return rc;
  if (p->dweight && (rc = check_matrix(p->dweight, p->dim, p->dweight_stride, "dweight", who))) return rc;
  const bool grad = p->dhidden || p->dweight;
  const Space s = space_of(p->n_rows, p->vocab, p->dim, p->piece_rows, grad);
  if (p->n_rows > 0) {
    if ((rc = check_matrix(p->hidden, p->dim, p->hidden_stride, "hidden", who))) return rc;
    if (p->dhidden && (rc = check_matrix(p->dhidden, p->dim, p->dhidden_stride, "dhidden", who))) return rc;
    if (!p->targets || !multiple_of(p->targets, 8)) return fail(ZERO_EINVAL, "%s: targets is NULL or misaligned", who);
    if (!p->logp || !multiple_of(p->logp, 4) || !multiple_of(p->row_weight, 4))
      return fail(ZERO_EINVAL, "%s: logp is NULL, or a per-row array is misaligned", who);
  }
  if (!p->workspace) return fail(ZERO_EINVAL, "%s: workspace is NULL", who);
  if (p->workspace_bytes < s.bytes)
    return fail(ZERO_EINVAL, "%s: workspace needs %llu bytes, got %zu", who, (unsigned long long)s.bytes, p->workspace_bytes);
  if (!multiple_of(p->workspace, 256)) return fail(ZERO_EINVAL, "%s: workspace must be 256-byte aligned", who);
  if ((rc = begin_launch())) return rc;
  char* ws = static_cast<char*>(p->workspace);
  HeadArgs a = {};
  a.weight = p->weight;
  a.hidden_stride = p->hidden_stride;
  a.weight_stride = p->weight_stride;
  a.vocab = p->vocab;
  a.dim = p->dim;
  a.tiles = s.tiles;
  a.shift = s.shift;
  a.padded = (p->vocab + 255) / 256 * 256;
  a.inv_temperature = 1.0 / p->temperature;
  a.coef = p->grad_scale / (p->divisor * p->temperature);
  a.c = (float)(kLog2e / p->temperature);
  a.dweight = p->dweight;
  a.dhidden_stride = p->dhidden_stride;
  a.dweight_stride = p->dweight_stride;
  a.meta = reinterpret_cast<Meta*>(ws + s.meta);
  a.row_of = reinterpret_cast<uint32_t*>(ws + s.row_of);
  a.target = reinterpret_cast<uint32_t*>(ws + s.target);
  a.omega = reinterpret_cast<float*>(ws + s.omega);
  a.said = reinterpret_cast<float*>(ws + s.said);
  a.rest = a.low = reinterpret_cast<float*>(ws + s.rest);
  if (grad && p->dtype == ZERO_F16 && p->row_weight) {
    a.lift = reinterpret_cast<float*>(ws + s.lift);
    a.low = reinterpret_cast<float*>(ws + s.low);
  }
  a.kept = reinterpret_cast<uint16_t*>(ws + s.kept);
  a.stats = reinterpret_cast<f32x2*>(ws + s.stats);
  a.held = reinterpret_cast<uint16_t*>(ws + s.held);
  a.part = reinterpret_cast<float*>(ws + s.part);
  a.sum = reinterpret_cast<float*>(ws + s.sum);
  double* terms = reinterpret_cast<double*>(ws + s.terms);
  uint8_t* counts = reinterpret_cast<uint8_t*>(ws + s.counts);
  // without rows, one empty piece: dweight is then zero
  uint64_t row = 0;
  do {
    a.rows = (uint32_t)std::min<uint64_t>(s.piece, p->n_rows - row);
    a.first = row == 0;
    a.last = row + a.rows == p->n_rows;
    a.planes = grad ? planes_of(a.rows, a.dim) : 1;
    a.hidden = static_cast<const uint16_t*>(p->hidden) + row * p->hidden_stride;
    a.targets = p->targets + row;
    a.row_weight = p->row_weight ? p->row_weight + row : nullptr;
    a.logp = p->logp + row;
    a.dhidden = p->dhidden ? static_cast<uint16_t*>(p->dhidden) + row * p->dhidden_stride : nullptr;
    a.terms = terms + row;
    a.counts = counts + row;
    if (a.rows > 0) {
      if (p->dtype == ZERO_F16) launch_piece<ZERO_F16>(a, grad, stream);
      else launch_piece<ZERO_BF16>(a, grad, stream);
    } else if (a.dweight) {
      hipLaunchKernelGGL(prepare_kernel, 1, 1024, 0, stream, a);
      if (p->dtype == ZERO_F16) launch_dweight<ZERO_F16>(a, stream);
      else launch_dweight<ZERO_BF16>(a, stream);
    }
    if ((rc = launch_status(who))) return rc;
    row += a.rows;
  } while (row < p->n_rows);
  hipLaunchKernelGGL(loss_kernel, 1, kBlock, 0, stream, terms, counts, p->n_rows, 1.0 / p->divisor, p->stats);
  return launch_status(who);
}
