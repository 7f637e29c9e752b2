// The owner step with both Adam moments in 8 bits, and the moments' way in and
// out of that form.
//
// State.  128 consecutive flat elements (an aligned block) share one fp32
// scale per moment.  The first moment is held as m ~ ms * m8, the second as
// its root, sqrt(v) ~ rs * r8, with m8 and r8 in e4m3 and the scale such that
// the block's largest magnitude is the format's largest value, 448.  Holding
// the root halves the exponent range that v needs, and the update divides by
// the root anyway.  e4m3 keeps 4 significant bits down to 2^-15 of the block's
// largest value and a step of 2^-18 below, so one block may span tensors of
// very different scale.  A block's largest element is exact up to its scale's
// fp32 rounding, so it decays as in 32 bits, and the rest keep their ratio to
// it.  A root above zero is never rounded to zero (it takes the smallest
// code): the update would otherwise divide its m by eps alone.
//
// The new weight is computed from the new fp32 moments, before they are
// rounded to 8 bits; the rounding only reaches the next step.  A non-finite
// gradient makes its block's scales NaN, and with them the block's moments: run
// the overflow check first where that can happen.
//
// Work.  One thread takes 8 flat elements, so 16 lanes (one DPP row) hold a
// block and its two maxima are four DPP steps each.  One 256-thread block
// takes one piece of the piece table: up to 2048 flat elements cut at flat
// multiples of 2048.  A piece that holds padding, or the owner's ragged end,
// has one mask byte per 8 elements; vectors with all bits set run like a
// whole piece's, the others element by element.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

#include "internal.h"
#include "launch.h"
#include "vec.h"

namespace zs {
namespace {

constexpr uint32_t kQBlock = ZERO_QBLOCK;
constexpr uint32_t kPiece = ZERO_PIECE;
constexpr uint32_t kMaskBytes = kPiece / 8;
constexpr float kCodeMax = 448.0f;             // largest e4m3 value
constexpr float kCodeTiny = 0x1p-9f;           // smallest positive one
constexpr float kLiveMin = 0x1p-100f;          // a block whose maximum is below this holds zeros:
                                               // 448 / maximum stays finite above it
static_assert(kPiece == 8 * kBlock && kQBlock == 8 * 16, "one vector per thread, one DPP row per block");

// ---------------------------------------------------------------------------
// A thread's eight elements.
// ---------------------------------------------------------------------------

// The real elements among [f, f + 8) of a piece, as a bit mask: the table's
// mask byte (all eight in a whole piece) within the piece and [begin, end).
__device__ __forceinline__ uint32_t real_bits(const zero_piece& pc, const uint8_t* masks, uint64_t n_masks,
                                              uint64_t begin, uint64_t end, uint64_t local_base, uint32_t t) {
  if (pc.flat % kQBlock != 0 || pc.flat < local_base || 8 * t >= pc.len || pc.len > kPiece) return 0;
  uint32_t bits = 0xFFu;
  if (pc.mask != ZERO_PIECE_WHOLE) {
    if (pc.mask >= n_masks) return 0;
    bits = masks[(uint64_t)pc.mask * kMaskBytes + t];
  }
  const uint64_t f = pc.flat + 8 * t;
  if (f < begin) bits &= f + 8 <= begin ? 0u : 0xFFu << (begin - f);
  if (f + 8 > end) bits &= f >= end ? 0u : 0xFFu >> (8 - (end - f));
  return bits & 0xFFu;
}

// fp32 values at index e: whole vectors as two 16-byte accesses, partial ones
// element by element (elements not real are neither read nor written).
template <int DT, bool NT = false>
__device__ __forceinline__ void get8(const void* p, uint64_t e, uint32_t bits, float (&x)[8]) {
  if (bits == 0xFFu) {
    const auto raw = load8<DT, NT>(p, e);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = Vec<DT>::get(raw, k);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = (bits >> k & 1) ? Vec<DT>::load1(p, e + k) : 0.0f;
  }
}

template <int DT, bool NT = false>
__device__ __forceinline__ void put8(void* p, uint64_t e, uint32_t bits, const float (&x)[8]) {
  if (bits == 0xFFu) {
    store8<DT, NT>(p, e, x);
    return;
  }
#pragma unroll
  for (int h = 0; h < 8; h += 4) {  // half a vector at a time where that is real
    const uint32_t half = bits >> h & 0xFu;
    if (half == 0xFu) {
      store4<DT>(p, e + h, x[h], x[h + 1], x[h + 2], x[h + 3]);
    } else if (half) {
#pragma unroll
      for (int k = h; k < h + 4; ++k)
        if (bits >> k & 1) Vec<DT>::store1(p, e + k, x[k]);
    }
  }
}

// Largest of a DPP row's 16 values, in every lane of it.
template <int CTRL>
__device__ __forceinline__ uint32_t row_max_step(uint32_t x) {
  return max(x, (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  x = row_max_step<0x128>(x);  // row_ror:8, 4, 2, 1
  x = row_max_step<0x124>(x);
  x = row_max_step<0x122>(x);
  return row_max_step<0x121>(x);
}

// Encodes the row's block: this thread's eight codes and the block's scale.
// The maximum is taken over magnitude bits, where NaN is largest.  A maximum
// that is not finite makes the scale NaN, so that every code decodes to NaN.
template <bool ROOT>
__device__ __forceinline__ u32x2 quantise(const float (&x)[8], float* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(x[k]) & 0x7FFFFFFFu);
  const float m = __uint_as_float(row_max(top));
  const bool dead = m < kLiveMin;  // false for NaN
  const float inv = dead ? 0.0f : kCodeMax * (1.0f / m);
  *scale = dead ? 0.0f : m * (1.0f / kCodeMax) + (m - m);
  float q[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    q[k] = x[k] * inv;
    if (ROOT) q[k] = x[k] > 0.0f && !dead ? fmaxf(q[k], kCodeTiny) : q[k];
  }
  return encode8(q);
}

struct Moments8 {
  uint8_t *m8, *r8;
  float *ms, *rs;
};

// The two moments of a thread's eight elements, as fp32 m and root.
__device__ __forceinline__ void load_moments(const Moments8& s, uint64_t l, float (&m)[8], float (&r)[8]) {
  const u32x2 cm = *reinterpret_cast<const u32x2*>(s.m8 + l), cr = *reinterpret_cast<const u32x2*>(s.r8 + l);
  const float ms = s.ms[l / kQBlock], rs = s.rs[l / kQBlock];
  decode8(cm, m);
  decode8(cr, r);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    m[k] = m[k] * ms;
    r[k] = r[k] * rs;
  }
}

// Encodes and stores them.  Every lane of the wavefront calls it.  Vectors
// without a real element are not written; the codes of padding inside a
// written vector are 0.
__device__ __forceinline__ void store_moments(const Moments8& s, uint64_t l, uint32_t bits, const float (&m)[8],
                                              const float (&r)[8]) {
  float ms, rs;
  const u32x2 cm = quantise<false>(m, &ms), cr = quantise<true>(r, &rs);
  const uint32_t row_any = row_max(bits);
  if (bits) {
    *reinterpret_cast<u32x2*>(s.m8 + l) = cm;
    *reinterpret_cast<u32x2*>(s.r8 + l) = cr;
  }
  if ((threadIdx.x & 15) == 0 && row_any) {
    s.ms[l / kQBlock] = ms;
    s.rs[l / kQBlock] = rs;
  }
}

// ---------------------------------------------------------------------------
// The step.
// ---------------------------------------------------------------------------
struct Ranks8 {
  const void* ptr[ZERO_MAX_RANKS];
  uint32_t R;
  uint64_t base;
  float divisor, inv_divisor;
  int32_t div_pow2;
};

struct Adam8Const {
  float beta1, one_minus_beta1, beta2, one_minus_beta2;
  float step_size;     // lr / (1 - beta1^t)
  float inv_sqrt_bc2;  // 1 / sqrt(1 - beta2^t)
  float eps;
  float decay;  // 1 - lr * wd for AdamW, else 1
  float l2;     // wd for classic Adam, else 0
  float clip;
};

struct Step8Args {
  Ranks8 rs;
  const zero_piece* pieces;
  uint64_t n_pieces;
  const uint8_t* masks;
  uint64_t n_masks;
  uint64_t begin, end;
  const float* reduced_g;
  float* w;
  Moments8 s;
  uint64_t local_base;
  void* p16;
  uint64_t param_base;
  Adam8Const c;
  uint32_t run;  // consecutive pieces to an XCD
};

// Gradient source, fixed at compile time:
//   RC > 0  : exactly RC rank buffers, all loads in flight together;
//   RC == 0 : any number of rank buffers, four in flight;
//   RC == kStored : a stored owner-local fp32 gradient.
constexpr int kStored = -1;

// The rank mean: ranks added in order from +0, one fp32 add each, then one IEEE
// division (a product with the exact reciprocal of a power of two).
__device__ __forceinline__ void mean(float (&g)[8], const Ranks8& rs) {
  if (rs.div_pow2) {
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = g[k] * rs.inv_divisor;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = g[k] / rs.divisor;
  }
}

template <int GDT>
__device__ __forceinline__ void add8(float (&g)[8], const typename Vec<GDT>::Raw& x) {
#pragma unroll
  for (int k = 0; k < 8; ++k) g[k] = g[k] + Vec<GDT>::get(x, k);
}

// sqrt(beta2 r^2 + (1 - beta2) g^2) where the sum is beyond fp32 and the root is
// not (g past 6e20 with beta2 = 0.999): the same with both scaled by a power of two.
__device__ __forceinline__ float large_root(const Adam8Const& c, float g, float r) {
  const float gs = g * 0x1p-66f, rs = r * 0x1p-66f;
  return __builtin_sqrtf((c.beta2 * rs) * rs + (c.one_minus_beta2 * gs) * gs) * 0x1p66f;
}

// The step on eight elements in registers.  m and v round after every
// operation: what a code's rounding turns on is then the same in any program
// that evaluates the formula in fp32.
__device__ __forceinline__ void adam8(const Adam8Const& c, const float (&g)[8], float (&w)[8], float (&m)[8],
                                      float (&r)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float gc = g[k] * c.clip;
    if (c.l2 != 0.0f) gc = fmaf(c.l2, w[k], gc);
    const float mn = c.beta1 * m[k] + c.one_minus_beta1 * gc;
    const float v = (c.beta2 * r[k]) * r[k] + (c.one_minus_beta2 * gc) * gc;
    float rn = __builtin_sqrtf(v);
    if (__builtin_expect(v == INFINITY, 0)) rn = large_root(c, gc, r[k]);
    const float denom = fmaf(rn, c.inv_sqrt_bc2, c.eps);
    w[k] = fmaf(-c.step_size, mn / denom, w[k] * c.decay);
    m[k] = mn;
    r[k] = rn;
  }
}

// Eight elements that lie inside every buffer, as vectors: every load is issued
// before the first is used.
template <int GDT, int RC>
__device__ __forceinline__ void load_vectors(const Step8Args& a, uint64_t f, float (&g)[8], float (&w)[8],
                                             float (&m)[8], float (&r)[8]) {
  constexpr bool kStream = GDT != ZERO_F32;  // 16-bit rank data is read once: nontemporal
  constexpr int kBatch = RC > 0 ? RC : 4;
  const uint64_t l = f - a.local_base;
  typename Vec<GDT>::Raw x[RC == kStored ? 1 : kBatch];
  if constexpr (RC == kStored) {
    x[0] = load8<GDT>(a.reduced_g, l);
  } else {
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (RC > 0 || (uint32_t)j < a.rs.R) x[j] = load8<GDT, kStream>(a.rs.ptr[j], f - a.rs.base);
  }
  const u32x2 cm = *reinterpret_cast<const u32x2*>(a.s.m8 + l), cr = *reinterpret_cast<const u32x2*>(a.s.r8 + l);
  const float ms = a.s.ms[l / kQBlock], rs = a.s.rs[l / kQBlock];
  const auto xw = load8<ZERO_F32>(a.w, l);
  __builtin_amdgcn_sched_barrier(0);  // no load sinks below the adds
  if constexpr (RC == kStored) {
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = Vec<GDT>::get(x[0], k);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = 0.0f;
    if constexpr (RC > 0) {
#pragma unroll
      for (int j = 0; j < RC; ++j) add8<GDT>(g, x[j]);
    } else {
      for (uint32_t r0 = 0; r0 < a.rs.R; r0 += kBatch) {
        typename Vec<GDT>::Raw y[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)  // the next four, while these are added
          if (r0 + kBatch + j < a.rs.R) y[j] = load8<GDT, kStream>(a.rs.ptr[r0 + kBatch + j], f - a.rs.base);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (r0 + j < a.rs.R) add8<GDT>(g, x[j]);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) x[j] = y[j];
      }
    }
    mean(g, a.rs);
  }
  decode8(cm, m);
  decode8(cr, r);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    w[k] = Vec<ZERO_F32>::get(xw, k);
    m[k] = m[k] * ms;
    r[k] = r[k] * rs;
  }
}

// The same element by element, for the vector that the buffers' end cuts.
template <int GDT, int RC>
__device__ __forceinline__ void load_elements(const Step8Args& a, uint64_t f, uint32_t bits, float (&g)[8],
                                              float (&w)[8], float (&m)[8], float (&r)[8]) {
  const uint64_t l = f - a.local_base;
  load_moments(a.s, l, m, r);
  get8<ZERO_F32>(a.w, l, bits, w);
  if constexpr (RC == kStored) {
    get8<ZERO_F32>(a.reduced_g, l, bits, g);
  } else {
    for (uint32_t j = 0; j < a.rs.R; ++j) {
      float x[8];
      get8<GDT>(a.rs.ptr[j], f - a.rs.base, bits, x);
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] = g[k] + x[k];
    }
    mean(g, a.rs);
  }
}

// A thread's eight elements of a piece; `bits` are the real ones (all of them
// in a WHOLE piece).  Padding beside real elements is loaded with them and
// then left out: it lies inside the buffers, and a vector at a time keeps
// every load of the wavefront in flight together (200,000 tensors of 100
// elements: 45 us element by element, 27 so).
template <int GDT, int PDT, int RC, bool WHOLE>
__device__ __forceinline__ void step_vector(const Step8Args& a, uint64_t f, uint32_t bits) {
  const uint64_t l = f - a.local_base;
  float g[8] = {}, w[8], m[8] = {}, r[8] = {};
  if (WHOLE || bits) {
    if (WHOLE || f + 8 <= a.end) load_vectors<GDT, RC>(a, f, g, w, m, r);
    else load_elements<GDT, RC>(a, f, bits, g, w, m, r);
    adam8(a.c, g, w, m, r);
    if constexpr (!WHOLE) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m[k] = (bits >> k & 1) ? m[k] : 0.0f;
        r[k] = (bits >> k & 1) ? r[k] : 0.0f;
      }
    }
    put8<ZERO_F32>(a.w, l, WHOLE ? 0xFFu : bits, w);
    if constexpr (PDT != ZERO_NONE) put8<PDT, true>(a.p16, f - a.param_base, WHOLE ? 0xFFu : bits, w);
  }
  store_moments(a.s, l, WHOLE ? 0xFFu : bits, m, r);
}

__device__ __forceinline__ bool is_whole(const zero_piece& pc, uint64_t begin, uint64_t end) {
  return pc.mask == ZERO_PIECE_WHOLE && pc.len == kPiece && pc.flat % kQBlock == 0 && pc.flat >= begin &&
         pc.flat <= end && end - pc.flat >= kPiece;
}

template <int GDT, int PDT, int RC>
__global__ void __launch_bounds__(kBlock) step8_kernel(const Step8Args a) {
  const uint32_t t = threadIdx.x;
  for (uint64_t i = xcd_runs(blockIdx.x, gridDim.x, a.run); i < a.n_pieces; i += gridDim.x) {
    const zero_piece pc = a.pieces[i];
    if (is_whole(pc, a.begin, a.end))
      step_vector<GDT, PDT, RC, true>(a, pc.flat + 8 * t, 0xFFu);
    else
      step_vector<GDT, PDT, RC, false>(a, pc.flat + 8 * t,
                                       real_bits(pc, a.masks, a.n_masks, a.begin, a.end, a.local_base, t));
  }
}

// ---------------------------------------------------------------------------
// fp32 moments to 8 bits and back.
// ---------------------------------------------------------------------------
struct Convert8Args {
  const zero_piece* pieces;
  uint64_t n_pieces;
  const uint8_t* masks;
  uint64_t n_masks;
  uint64_t begin, end, local_base;
  float *m, *v;  // fp32 moments, owner-local
  Moments8 s;
};

template <bool PACK>
__global__ void __launch_bounds__(kBlock) convert8_kernel(const Convert8Args a) {
  const uint32_t t = threadIdx.x;
  for (uint64_t i = blockIdx.x; i < a.n_pieces; i += gridDim.x) {
    const zero_piece pc = a.pieces[i];
    const uint32_t bits = real_bits(pc, a.masks, a.n_masks, a.begin, a.end, a.local_base, t);
    const uint64_t l = pc.flat + 8 * t - a.local_base;
    float m[8] = {}, r[8] = {};
    if constexpr (PACK) {
      if (bits) {
        // as vectors unless the buffers' end cuts them, then without the padding
        const uint32_t in = pc.flat + 8 * t + 8 <= a.end ? 0xFFu : bits;
        get8<ZERO_F32>(a.m, l, in, m);
        get8<ZERO_F32>(a.v, l, in, r);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          m[k] = (bits >> k & 1) ? m[k] : 0.0f;
          r[k] = (bits >> k & 1) ? __builtin_sqrtf(r[k]) : 0.0f;
        }
      }
      store_moments(a.s, l, bits, m, r);
    } else if (bits) {
      load_moments(a.s, l, m, r);
#pragma unroll
      for (int k = 0; k < 8; ++k) r[k] = r[k] * r[k];
      put8<ZERO_F32>(a.m, l, bits, m);
      put8<ZERO_F32>(a.v, l, bits, r);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side: validation and launch.
// ---------------------------------------------------------------------------
bool exact_reciprocal(float d, float* inv) {
  int e = 0;
  if (std::frexp(d, &e) != 0.5f) return false;
  const float r = std::ldexp(1.0f, 1 - e);
  if (!std::isnormal(r)) return false;
  *inv = r;
  return true;
}

int fill_ranks8(Ranks8* rs, const zero_adam8_args* p, const char* who) {
  if (p->R == 0 || p->R > ZERO_MAX_RANKS)
    return fail(ZERO_EINVAL, "%s: R = %u outside [1, %d]", who, p->R, ZERO_MAX_RANKS);
  if (!p->rank_grads) return fail(ZERO_EINVAL, "%s: neither rank_grads nor reduced_g is given", who);
  if (p->grad_dtype != ZERO_F16 && p->grad_dtype != ZERO_BF16 && p->grad_dtype != ZERO_F32)
    return fail(ZERO_EINVAL, "%s: unknown gradient dtype %d", who, p->grad_dtype);
  if (p->grad_base % 8 != 0 || p->grad_base > p->begin)
    return fail(ZERO_EINVAL, "%s: grad_base must be a multiple of 8 and <= begin", who);
  if (!(p->divisor > 0.0f) || !std::isfinite(p->divisor))
    return fail(ZERO_EINVAL, "%s: divisor must be finite and > 0", who);
  for (uint32_t r = 0; r < p->R; ++r) {
    if (!p->rank_grads[r]) return fail(ZERO_EINVAL, "%s: rank buffer %u is NULL", who, r);
    if (!aligned16(p->rank_grads[r]))
      return fail(ZERO_EINVAL, "%s: rank buffer %u is not 16-byte aligned", who, r);
    rs->ptr[r] = p->rank_grads[r];
  }
  rs->R = p->R;
  rs->base = p->grad_base;
  rs->divisor = p->divisor;
  rs->div_pow2 = exact_reciprocal(p->divisor, &rs->inv_divisor) ? 1 : 0;
  return ZERO_OK;
}

// The piece table, owner range and 8-bit state that every call here takes.
int check_state8(const zero_piece* pieces, uint64_t n_pieces, const uint8_t* masks, uint64_t n_masks, uint64_t begin,
                 uint64_t end, uint64_t local_base, const Moments8& s, const char* who) {
  if (begin > end) return fail(ZERO_EINVAL, "%s: begin > end", who);
  if (n_pieces > 0 && !pieces) return fail(ZERO_EINVAL, "%s: pieces is NULL", who);
  if (n_masks > 0 && !masks) return fail(ZERO_EINVAL, "%s: masks is NULL", who);
  if (local_base % kQBlock != 0 || local_base > begin)
    return fail(ZERO_EINVAL, "%s: local_base must be a multiple of %u and <= begin", who, kQBlock);
  if (!s.m8 || !s.r8 || !s.ms || !s.rs) return fail(ZERO_EINVAL, "%s: the 8-bit state arrays must be given", who);
  if (!aligned16(s.m8) || !aligned16(s.r8) || !aligned16(s.ms) || !aligned16(s.rs))
    return fail(ZERO_EINVAL, "%s: state arrays must be 16-byte aligned", who);
  return ZERO_OK;
}

template <int GDT, int RC>
void launch_step8_p(Step8Args& a, int pdt, hipStream_t s) {
  const uint32_t grid = chunk_grid(a.n_pieces, 0);
  // Whole pieces: at most three blocks to a CU, four with up to five 16-bit
  // rank buffers, whose loads are fewer, and runs of two pieces to an XCD.
  // 8 bf16 ranks into 1.0e8 elements: 512 us; two blocks 562, four 533,
  // uncapped 538, single pieces 516.  4 bf16 ranks into 6e7 elements: 226 us;
  // three blocks 229, uncapped 230; 1 rank 184; three 194, uncapped 178.  The
  // stored gradient goes by single pieces: 3.75e8 elements 1118 us, in runs
  // 1147 (and so 1479 with two blocks, 1221 with four, 1259 uncapped).  Pieces
  // with padding wait for more round trips and want every block that fits:
  // 200,000 tensors of 100 elements 27.4 us, 29.0 with four blocks.
  const bool whole = 2 * a.n_masks <= a.n_pieces;
  const bool light = GDT != ZERO_F32 && a.rs.R <= 5;
  const uint32_t lds = whole ? lds_for_blocks_per_cu(light ? 4 : 3, 0) : 0;
  a.run = whole && RC != kStored ? 2 : 1;
  if (pdt == ZERO_F16) hipLaunchKernelGGL((step8_kernel<GDT, ZERO_F16, RC>), grid, kBlock, lds, s, a);
  else if (pdt == ZERO_BF16) hipLaunchKernelGGL((step8_kernel<GDT, ZERO_BF16, RC>), grid, kBlock, lds, s, a);
  else hipLaunchKernelGGL((step8_kernel<GDT, ZERO_NONE, RC>), grid, kBlock, lds, s, a);
}

// Up to eight ranks have all their loads unrolled; more take four at a time
// (taking 3 or 5 ranks so as well cost 15% and 7%).
template <int GDT>
void launch_step8(Step8Args& a, int pdt, hipStream_t s) {
  switch (a.rs.R) {
    case 1: return launch_step8_p<GDT, 1>(a, pdt, s);
    case 2: return launch_step8_p<GDT, 2>(a, pdt, s);
    case 3: return launch_step8_p<GDT, 3>(a, pdt, s);
    case 4: return launch_step8_p<GDT, 4>(a, pdt, s);
    case 5: return launch_step8_p<GDT, 5>(a, pdt, s);
    case 6: return launch_step8_p<GDT, 6>(a, pdt, s);
    case 7: return launch_step8_p<GDT, 7>(a, pdt, s);
    case 8: return launch_step8_p<GDT, 8>(a, pdt, s);
    default: return launch_step8_p<GDT, 0>(a, pdt, s);
  }
}

int convert8(bool pack, const zero_piece* pieces, uint64_t n_pieces, const uint8_t* masks, uint64_t n_masks,
             uint64_t begin, uint64_t end, uint64_t local_base, float* m, float* v, const Moments8& s,
             hipStream_t stream, const char* who) {
  clear_error();
  int rc = check_state8(pieces, n_pieces, masks, n_masks, begin, end, local_base, s, who);
  if (rc) return rc;
  if (!m || !v) return fail(ZERO_EINVAL, "%s: exp_avg and exp_avg_sq must be given", who);
  if (!aligned16(m) || !aligned16(v)) return fail(ZERO_EINVAL, "%s: state arrays must be 16-byte aligned", who);
  if (n_pieces == 0 || begin == end) return ZERO_OK;
  if ((rc = begin_launch())) return rc;
  const Convert8Args a = {pieces, n_pieces, masks, n_masks, begin, end, local_base, m, v, s};
  const uint32_t grid = chunk_grid(n_pieces, 0);
  if (pack) hipLaunchKernelGGL(convert8_kernel<true>, grid, kBlock, 0, stream, a);
  else hipLaunchKernelGGL(convert8_kernel<false>, grid, kBlock, 0, stream, a);
  return launch_status(who);
}

}  // namespace
}  // namespace zs

using namespace zs;

extern "C" int zero_adam8_step(const zero_adam8_args* p, hipStream_t stream) {
  static const char* who = "zero_adam8_step";
  clear_error();
  if (!p) return fail(ZERO_EINVAL, "%s: args is NULL", who);
  if (p->step == 0) return fail(ZERO_EINVAL, "%s: step counts from 1", who);
  Step8Args a;
  std::memset(&a, 0, sizeof a);
  a.s = {p->exp_avg8, p->exp_rms8, p->exp_avg_scale, p->exp_rms_scale};
  int rc = check_state8(p->pieces, p->n_pieces, p->masks, p->n_masks, p->begin, p->end, p->local_base, a.s, who);
  if (rc) return rc;
  if (p->reduced_g) {
    if (!aligned16(p->reduced_g)) return fail(ZERO_EINVAL, "%s: reduced_g is not 16-byte aligned", who);
  } else if ((rc = fill_ranks8(&a.rs, p, who))) {
    return rc;
  }
  if (!p->master) return fail(ZERO_EINVAL, "%s: master must be given", who);
  if (!aligned16(p->master)) return fail(ZERO_EINVAL, "%s: master is not 16-byte aligned", who);
  const int pdt = p->param_dtype;
  if (pdt != ZERO_NONE && pdt != ZERO_F16 && pdt != ZERO_BF16)
    return fail(ZERO_EINVAL, "%s: param_dtype must be NONE, F16 or BF16", who);
  if (pdt != ZERO_NONE) {
    if (!p->param16) return fail(ZERO_EINVAL, "%s: param16 is NULL", who);
    if (!aligned16(p->param16)) return fail(ZERO_EINVAL, "%s: param16 is not 16-byte aligned", who);
    if (p->param_base % 8 != 0 || p->param_base > p->begin)
      return fail(ZERO_EINVAL, "%s: param_base must be a multiple of 8 and <= begin", who);
  }
  const double hp[] = {p->lr, p->beta1, p->beta2, p->eps, p->weight_decay, p->clip_coef};
  for (double x : hp)
    if (!std::isfinite(x)) return fail(ZERO_EINVAL, "%s: non-finite hyperparameter", who);
  if (p->lr < 0 || p->eps < 0 || p->weight_decay < 0 || p->clip_coef < 0)
    return fail(ZERO_EINVAL, "%s: lr, eps, weight_decay and clip_coef must be >= 0", who);
  if (p->beta1 < 0 || p->beta1 >= 1 || p->beta2 < 0 || p->beta2 >= 1)
    return fail(ZERO_EINVAL, "%s: betas must lie in [0, 1)", who);
  if (p->n_pieces == 0 || p->begin == p->end) return ZERO_OK;
  if ((rc = begin_launch())) return rc;

  // Constants in fp64, each rounded once to fp32.
  const double t = (double)p->step;
  a.c.beta1 = (float)p->beta1;
  a.c.one_minus_beta1 = (float)(1.0 - p->beta1);
  a.c.beta2 = (float)p->beta2;
  a.c.one_minus_beta2 = (float)(1.0 - p->beta2);
  a.c.step_size = (float)(p->lr / (1.0 - std::pow(p->beta1, t)));
  a.c.inv_sqrt_bc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(p->beta2, t)));
  a.c.eps = (float)p->eps;
  a.c.decay = p->adamw ? (float)(1.0 - p->lr * p->weight_decay) : 1.0f;
  a.c.l2 = p->adamw ? 0.0f : (float)p->weight_decay;
  a.c.clip = (float)p->clip_coef;
  a.pieces = p->pieces;
  a.n_pieces = p->n_pieces;
  a.masks = p->masks;
  a.n_masks = p->n_masks;
  a.begin = p->begin;
  a.end = p->end;
  a.reduced_g = p->reduced_g;
  a.w = p->master;
  a.local_base = p->local_base;
  a.p16 = pdt != ZERO_NONE ? p->param16 : nullptr;
  a.param_base = p->param_base;
  if (p->reduced_g) launch_step8_p<ZERO_F32, kStored>(a, pdt, stream);
  else if (p->grad_dtype == ZERO_F16) launch_step8<ZERO_F16>(a, pdt, stream);
  else if (p->grad_dtype == ZERO_BF16) launch_step8<ZERO_BF16>(a, pdt, stream);
  else launch_step8<ZERO_F32>(a, pdt, stream);
  return launch_status(who);
}

extern "C" int zero_moments8_pack(const zero_piece* pieces, uint64_t n_pieces, const uint8_t* masks, uint64_t n_masks,
                                  uint64_t begin, uint64_t end, uint64_t local_base, const float* exp_avg,
                                  const float* exp_avg_sq, uint8_t* exp_avg8, float* exp_avg_scale, uint8_t* exp_rms8,
                                  float* exp_rms_scale, hipStream_t stream) {
  return convert8(true, pieces, n_pieces, masks, n_masks, begin, end, local_base, const_cast<float*>(exp_avg),
                  const_cast<float*>(exp_avg_sq), Moments8{exp_avg8, exp_rms8, exp_avg_scale, exp_rms_scale}, stream,
                  "zero_moments8_pack");
}

extern "C" int zero_moments8_unpack(const zero_piece* pieces, uint64_t n_pieces, const uint8_t* masks,
                                    uint64_t n_masks, uint64_t begin, uint64_t end, uint64_t local_base,
                                    const uint8_t* exp_avg8, const float* exp_avg_scale, const uint8_t* exp_rms8,
                                    const float* exp_rms_scale, float* exp_avg, float* exp_avg_sq,
                                    hipStream_t stream) {
  return convert8(false, pieces, n_pieces, masks, n_masks, begin, end, local_base, exp_avg, exp_avg_sq,
                  Moments8{const_cast<uint8_t*>(exp_avg8), const_cast<uint8_t*>(exp_rms8),
                           const_cast<float*>(exp_avg_scale), const_cast<float*>(exp_rms_scale)},
                  stream, "zero_moments8_unpack");
}
