// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[n]    = scale table[token[n]]            (0 for a token outside the table)
//   dtable[v] = scale sum of dout[n] over the n with token[n] = v, n ascending
//
// Both are bound by HBM: the lookup reads and writes each row once; the
// gradient reads dout once and writes the table once (or, added onto another
// gradient, reads and writes the rows that tokens name).  The sum over equal
// tokens has a fixed order, so tokens are sorted (a stable radix sort of
// (token, position), whole numbers only) and no float is added atomically.
// 16,384 tokens of 128,000 x 4096 bf16: lookup 42 us (6.3 TB/s); gradient 258 us for
// 1.18 GB: the zeros 175, beside them the sort, the sums 72, the runs over several
// tiles 9.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "launch.h"
#include "rows.h"

namespace zs {
namespace {

// ---------------------------------------------------------------------------
// Lookup.
// ---------------------------------------------------------------------------
struct EmbedArgs {
  const void* table;
  const int64_t* tokens;
  void* out;
  uint64_t n_tokens, stride;  // stride: of the table's rows
  uint32_t vocab, dim, vecs;  // vecs: 16-byte vectors of a row
  float scale;
};

// 2^SH threads to a row, one vector each at a time.
template <int DT>
__global__ void __launch_bounds__(kBlock) embed_kernel(const EmbedArgs a, const uint32_t shift) {
  constexpr int N = Lane<DT>::N;
  typedef typename Vec<DT>::T T;
  const uint32_t lanes = 1u << shift, rows = kBlock >> shift;
  for (uint64_t n = (uint64_t)blockIdx.x * rows + (threadIdx.x >> shift); n < a.n_tokens; n += (uint64_t)gridDim.x * rows) {
    const int64_t token = a.tokens[n];
    const bool has = token >= 0 && token < (int64_t)a.vocab;
    const T* from = static_cast<const T*>(a.table) + (has ? (uint64_t)token * a.stride : 0);
    T* to = static_cast<T*>(a.out) + n * a.dim;
    for (uint32_t v = threadIdx.x & (lanes - 1); v < a.vecs; v += lanes) {
      float x[N] = {};
      if (has) {
        const u32x4 r = load_cut<DT>(from, v, a.dim);
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] = Lane<DT>::get(r, k) * a.scale;
      }
      store_cut<DT>(to, v, a.dim, x);
    }
  }
}

// ---------------------------------------------------------------------------
// Stable radix sort of (token, position).
//
// A pass takes up to 9 bits.  Blocks of 256 threads take 2048 consecutive
// keys; a wavefront takes 512 of them in 8 rounds of 64.  In a round a lane
// finds the lanes with its digit by one ballot per bit, its rank among them by
// a population count, and the count so far in its wavefront's own counters:
// the order within a digit is the order of the keys.
// ---------------------------------------------------------------------------
constexpr uint32_t kSortKeys = 2048, kRounds = kSortKeys / kBlock, kMaxBits = 9, kDigits = 1u << kMaxBits;

struct SortArgs {
  const int64_t* tokens;      // the first pass reads these,
  const uint32_t *keys, *at;  // the others these
  uint32_t *keys_out, *at_out;
  uint32_t* hist;    // [1 << bits][blocks], of many blocks counts of the blocks before
  uint32_t* totals;  // [1 << bits], of many blocks
  uint32_t n, vocab, blocks, shift, bits;
};

// A token outside the table sorts behind all others.
__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, uint32_t i) {
  if (a.tokens) {
    const int64_t t = a.tokens[i];
    return t >= 0 && t < (int64_t)a.vocab ? (uint32_t)t : a.vocab;
  }
  return a.keys[i];
}

__global__ void __launch_bounds__(kBlock) histogram_kernel(const SortArgs a) {
  __shared__ uint32_t count[kDigits];
  const uint32_t digits = 1u << a.bits;
  for (uint32_t d = threadIdx.x; d < digits; d += kBlock) count[d] = 0;
  __syncthreads();
  const uint32_t begin = blockIdx.x * kSortKeys;
#pragma unroll
  for (uint32_t r = 0; r < kRounds; ++r) {
    const uint32_t i = begin + r * kBlock + threadIdx.x;
    if (i < a.n) atomicAdd(&count[sort_key(a, i) >> a.shift & (digits - 1)], 1u);
  }
  __syncthreads();
  for (uint32_t d = threadIdx.x; d < digits; d += kBlock) a.hist[(uint64_t)d * a.blocks + blockIdx.x] = count[d];
}

// Of many blocks: a digit's counts become those of the blocks before, one block to
// a digit.  (Few blocks add them up themselves: a launch less, and what they then
// read grows with their square.  Onto a gradient of 64 columns bf16, added up by
// themselves and scanned: 10 blocks 59 and 61 us, 20 blocks 73 and 69, 35 blocks 88 and
// 72, 64 blocks 121 and 100, 98 blocks 171 and 122, 489 blocks 811 and 409.)
constexpr uint32_t kScanBlocks = 16;
__global__ void __launch_bounds__(kBlock) scan_kernel(const SortArgs a) {
  __shared__ uint32_t sums[kWavesPerBlock];
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
  uint32_t* row = a.hist + (uint64_t)blockIdx.x * a.blocks;
  uint32_t before = 0;
  for (uint32_t b0 = 0; b0 < a.blocks; b0 += kBlock) {
    const uint32_t own = b0 + t < a.blocks ? row[b0 + t] : 0;
    uint32_t sum = own;
#pragma unroll
    for (uint32_t s = 1; s < 64; s <<= 1) {
      const uint32_t up = __shfl_up(sum, s, 64);
      if (lane >= s) sum += up;
    }
    __syncthreads();
    if (lane == 63) sums[wave] = sum;
    __syncthreads();
    for (uint32_t w = 0; w < wave; ++w) sum += sums[w];
    if (b0 + t < a.blocks) row[b0 + t] = before + sum - own;
#pragma unroll
    for (uint32_t w = 0; w < kWavesPerBlock; ++w) before += sums[w];
  }
  if (t == 0) a.totals[blockIdx.x] = before;
}

__global__ void __launch_bounds__(kBlock) scatter_kernel(const SortArgs a) {
  __shared__ uint32_t count[kWavesPerBlock][kDigits];  // of a wavefront, then where its keys of a digit begin
  __shared__ uint32_t sums[kWavesPerBlock];
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6, digits = 1u << a.bits;
  for (uint32_t d = t; d < kWavesPerBlock * kDigits; d += kBlock) (&count[0][0])[d] = 0;
  __syncthreads();
  uint32_t key[kRounds], rank[kRounds];
  const uint32_t begin = blockIdx.x * kSortKeys + wave * (kSortKeys / kWavesPerBlock) + lane;
#pragma unroll
  for (uint32_t r = 0; r < kRounds; ++r) {
    const uint32_t i = begin + r * 64;
    key[r] = i < a.n ? sort_key(a, i) : 0;
  }
#pragma unroll
  for (uint32_t r = 0; r < kRounds; ++r) {
    const bool has = begin + r * 64 < a.n;
    const uint32_t d = key[r] >> a.shift & (digits - 1);
    uint64_t same = __ballot(has);
    for (uint32_t b = 0; b < a.bits; ++b) {
      const uint64_t one = __ballot(d >> b & 1);
      same &= (d >> b & 1) ? one : ~one;
    }
    const uint32_t before = __popcll(same & ((1ull << lane) - 1));
    const uint32_t seen = count[wave][d];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (has && before == 0) count[wave][d] = seen + (uint32_t)__popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    rank[r] = seen + before;
  }
  __syncthreads();
  // Where each digit of this block begins: behind all smaller digits, and
  // behind the earlier blocks' keys of the same one.  A thread takes two
  // neighbouring digits.
  uint32_t total[2] = {0, 0}, mine[2] = {0, 0};
#pragma unroll
  for (uint32_t j = 0; j < 2; ++j) {
    const uint32_t d = 2 * t + j;
    if (d >= digits) continue;
    if (a.blocks > kScanBlocks) {
      mine[j] = a.hist[(uint64_t)d * a.blocks + blockIdx.x];
      total[j] = a.totals[d];
    } else
      for (uint32_t b = 0; b < a.blocks; ++b) {
        const uint32_t c = a.hist[(uint64_t)d * a.blocks + b];
        mine[j] += b < blockIdx.x ? c : 0;
        total[j] += c;
      }
  }
  uint32_t sum = total[0] + total[1];
#pragma unroll
  for (uint32_t s = 1; s < 64; s <<= 1) {
    const uint32_t up = __shfl_up(sum, s, 64);
    if (lane >= s) sum += up;
  }
  if (lane == 63) sums[wave] = sum;
  __syncthreads();
  for (uint32_t w = 0; w < wave; ++w) sum += sums[w];
  uint32_t start = sum - total[0] - total[1];
#pragma unroll
  for (uint32_t j = 0; j < 2; ++j) {
    const uint32_t d = 2 * t + j;
    if (d < digits) {
      uint32_t at = start + mine[j];
#pragma unroll
      for (int w = 0; w < kWavesPerBlock; ++w) {
        const uint32_t c = count[w][d];
        count[w][d] = at;
        at += c;
      }
    }
    start += total[j];
  }
  __syncthreads();
#pragma unroll
  for (uint32_t r = 0; r < kRounds; ++r) {
    const uint32_t i = begin + r * 64;
    if (i < a.n) {
      const uint32_t to = count[wave][key[r] >> a.shift & (digits - 1)] + rank[r];
      a.keys_out[to] = key[r];
      a.at_out[to] = a.tokens ? i : a.at[i];
    }
  }
}

// ---------------------------------------------------------------------------
// Sums over the sorted positions.
//
// They are cut into tiles of 8 or, from kFewTokens on, 32 (onto a gradient of 4096
// columns bf16: 4096 tokens 40 us with 8, 42 with 32; 8192 tokens 68 and 58).  A run of equal tokens that lies within a
// tile is summed and written there; one that a tile's end cuts leaves partial
// sums (fp32, of up to 32 rows), the tile's first run in slot 0, its last one in
// slot 1, which join_kernel adds in the order of the tiles.
// ---------------------------------------------------------------------------
constexpr uint32_t kFewTokens = 4096, kFewTile = 8, kTile = 32;

struct GradArgs {
  const uint32_t *keys, *at;  // sorted
  const void* dout;
  void* dtable;
  float* partial;  // [tiles][2][vecs * N]
  uint64_t stride;
  uint32_t n, vocab, dim, vecs, tile;
  float scale;
  bool accumulate;
};

// dtable's row `key`, vector v of dout's: as it is, in OUT's vectors.
template <int DT, int OUT>
struct Old {
  static constexpr int kVecs = DT == OUT ? 1 : 2;  // a 16-bit gradient into an fp32 table: two for one
  u32x4 q[kVecs];
  __device__ __forceinline__ void load(const void* row, uint32_t v, uint32_t dim) {
#pragma unroll
    for (int h = 0; h < kVecs; ++h) q[h] = load_cut<OUT>(row, v * kVecs + h, dim);
  }
  __device__ __forceinline__ float get(int k) const { return Lane<OUT>::get(q[k / Lane<OUT>::N], k % Lane<OUT>::N); }
};

template <int DT, int OUT>
__device__ __forceinline__ void write_row(const GradArgs& a, uint32_t key, uint32_t v, const float (&sum)[Lane<DT>::N],
                                          const Old<DT, OUT>& old) {
  constexpr int M = Lane<OUT>::N;
  typename Vec<OUT>::T* row = static_cast<typename Vec<OUT>::T*>(a.dtable) + (uint64_t)key * a.stride;
#pragma unroll
  for (int h = 0; h < Old<DT, OUT>::kVecs; ++h) {
    float x[M];
#pragma unroll
    for (int k = 0; k < M; ++k) {
      x[k] = sum[h * M + k] * a.scale;
      if (a.accumulate) x[k] += old.get(h * M + k);
    }
    store_cut<OUT>(row, v * Old<DT, OUT>::kVecs + h, a.dim, x);
  }
}

template <int DT, int OUT>
__global__ void __launch_bounds__(kBlock) sum_kernel(const GradArgs a) {
  constexpr int N = Lane<DT>::N;
  typedef typename Vec<DT>::T T;
  __shared__ uint32_t key[kTile + 2], at[kTile];
  const uint32_t begin = blockIdx.x * a.tile, end = min(begin + a.tile, a.n), n = end - begin;
  // key[0] and key[n + 1]: the neighbours' (a number that no key has, at the ends)
  for (uint32_t i = threadIdx.x; i < n + 2; i += kBlock) {
    const int64_t p = (int64_t)begin + i - 1;
    key[i] = p >= 0 && p < (int64_t)a.n ? a.keys[p] : 0xFFFFFFFFu;
    if (i >= 1 && i <= n) at[i - 1] = a.at[p];
  }
  __syncthreads();
  for (uint32_t v = blockIdx.y * kBlock + threadIdx.x; v < a.vecs; v += gridDim.y * kBlock) {
    float sum[N] = {};
    bool cut = key[0] == key[1];  // the run at hand began in an earlier tile
    constexpr uint32_t B = 8;     // rows in flight, and the rows they are added to
    for (uint32_t i0 = 0; i0 < n; i0 += B) {
      u32x4 r[B];
      Old<DT, OUT> old[B];
#pragma unroll
      for (uint32_t j = 0; j < B; ++j) {
        const uint32_t i = i0 + j;
        r[j] = u32x4{0, 0, 0, 0};
        if (i < n && key[i + 1] < a.vocab) {
          r[j] = load_cut<DT>(static_cast<const T*>(a.dout) + (uint64_t)at[i] * a.dim, v, a.dim);
          if (a.accumulate && key[i + 2] != key[i + 1])
            old[j].load(static_cast<typename Vec<OUT>::T*>(a.dtable) + (uint64_t)key[i + 1] * a.stride, v, a.dim);
        }
      }
#pragma unroll
      for (uint32_t j = 0; j < B; ++j) {
        const uint32_t i = i0 + j;
        if (i >= n) break;
        const uint32_t k0 = key[i + 1];
        if (k0 >= a.vocab) break;
#pragma unroll
        for (int k = 0; k < N; ++k) sum[k] += Lane<DT>::get(r[j], k);
        const bool last = key[i + 2] != k0;
        if (last && !cut) write_row<DT, OUT>(a, k0, v, sum, old[j]);
        else if (last || i + 1 == n) {
          f32x4* to = reinterpret_cast<f32x4*>(a.partial + (((uint64_t)blockIdx.x * 2 + (cut ? 0 : 1)) * a.vecs + v) * N);
#pragma unroll
          for (int k = 0; k < N; k += 4) to[k / 4] = f32x4{sum[k], sum[k + 1], sum[k + 2], sum[k + 3]};
        }
        if (last) {
          cut = false;
#pragma unroll
          for (int k = 0; k < N; ++k) sum[k] = 0.0f;
        }
      }
    }
  }
}

// The first position in [lo, hi] whose key is at least x (hi: none), for a whole wavefront.
__device__ __forceinline__ uint32_t first_at_least(const uint32_t* keys, uint32_t lo, uint32_t hi, uint32_t x) {
  const uint32_t lane = threadIdx.x & 63;
  while (hi > lo) {
    const uint32_t step = (hi - lo + 63) / 64, p = lo + lane * step;
    const uint32_t c = (uint32_t)__popcll(__ballot(p < hi && keys[p] < x));  // probes 0 .. c - 1 are below x
    if (c == 0) break;
    hi = min(hi, lo + c * step);
    lo += (c - 1) * step + 1;
  }
  return lo;
}

// Tile b's last run, where it began in the tile and goes on behind it.  The tiles'
// sums are added in fp64: a padding token that nothing masks has a run as long as
// the batch, and a chain of fp32 additions can be off in proportion to its length
// (150,000 rows of 1 + 2^-13: by 7e-5 of the sum; of random numbers of one sign 1.7e-6,
// with the tiles' sums in fp64 1.1e-7).
template <int DT, int OUT>
__global__ void __launch_bounds__(kBlock) join_kernel(const GradArgs a) {
  constexpr int N = Lane<DT>::N;
  const uint32_t begin = blockIdx.x * a.tile, end = begin + a.tile;
  if (end >= a.n) return;
  const uint32_t key = a.keys[end - 1];
  if (key >= a.vocab || a.keys[end] != key) return;   // ends here
  if (begin > 0 && a.keys[begin - 1] == key) return;  // began earlier
  const uint32_t last = (first_at_least(a.keys, end, a.n, key + 1) - 1) / a.tile;  // the run's last tile
  for (uint32_t v = blockIdx.y * kBlock + threadIdx.x; v < a.vecs; v += gridDim.y * kBlock) {
    double total[N];
    Old<DT, OUT> old;
    if (a.accumulate)
      old.load(static_cast<typename Vec<OUT>::T*>(a.dtable) + (uint64_t)key * a.stride, v, a.dim);
    const auto part = [&](uint32_t tile, uint32_t slot, int k) {
      return reinterpret_cast<const f32x4*>(a.partial + (((uint64_t)tile * 2 + slot) * a.vecs + v) * N)[k];
    };
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
      const f32x4 p = part(blockIdx.x, 1, k);
#pragma unroll
      for (int j = 0; j < 4; ++j) total[4 * k + j] = (double)p[j];
    }
    uint32_t b = blockIdx.x + 1;
    constexpr uint32_t B = 8;  // partial rows in flight
    for (; b + B <= last + 1; b += B) {
      f32x4 p[B][N / 4];
#pragma unroll
      for (uint32_t i = 0; i < B; ++i)
#pragma unroll
        for (int k = 0; k < N / 4; ++k) p[i][k] = part(b + i, 0, k);
#pragma unroll
      for (uint32_t i = 0; i < B; ++i)
#pragma unroll
        for (int k = 0; k < N; ++k) total[k] += (double)p[i][k / 4][k % 4];
    }
    for (; b <= last; ++b) {
#pragma unroll
      for (int k = 0; k < N / 4; ++k) {
        const f32x4 p = part(b, 0, k);
#pragma unroll
        for (int j = 0; j < 4; ++j) total[4 * k + j] += (double)p[j];
      }
    }
    float sum[N];
#pragma unroll
    for (int k = 0; k < N; ++k) sum[k] = (float)total[k];
    write_row<DT, OUT>(a, key, v, sum, old);
  }
}

// The rows of the table that no token names are zero.  A block takes kFillRows
// of them and finds the sorted keys of that range by bisection, 64 probes at a time.
constexpr uint32_t kFillRows = 16;

template <int OUT>
__global__ void __launch_bounds__(kBlock) fill_kernel(const GradArgs a, uint32_t vecs) {
  constexpr int N = Lane<OUT>::N;
  typedef typename Vec<OUT>::T T;
  __shared__ uint32_t named;
  const uint32_t lane = threadIdx.x & 63;
  for (uint32_t row0 = blockIdx.x * kFillRows; row0 < a.vocab; row0 += gridDim.x * kFillRows) {
    __syncthreads();
    if (threadIdx.x < 64) {
      uint32_t p = first_at_least(a.keys, 0, a.n, row0);
      uint32_t bits = 0;
      while (p < a.n) {
        const uint32_t k = p + lane < a.n ? a.keys[p + lane] : 0xFFFFFFFFu;
        if (k < row0 + kFillRows) bits |= 1u << (k - row0);
        if (__ballot(k >= row0 + kFillRows)) break;
        p += 64;
        const uint32_t last = (uint32_t)__builtin_amdgcn_readlane((int)k, 63);
        if ((uint32_t)__builtin_amdgcn_readfirstlane((int)k) == last) p = first_at_least(a.keys, p, a.n, last + 1);
      }
#pragma unroll
      for (uint32_t s = 1; s < 64; s <<= 1) bits |= (uint32_t)__shfl_xor((int)bits, s, 64);
      if (lane == 0) named = bits;
    }
    __syncthreads();
    const uint32_t skip = named, rows = min(kFillRows, a.vocab - row0);
    const float zero[N] = {};
    for (uint32_t r = 0; r < rows; ++r) {
      if (skip >> r & 1) continue;
      T* row = static_cast<T*>(a.dtable) + (uint64_t)(row0 + r) * a.stride;
      for (uint32_t v = threadIdx.x; v < vecs; v += kBlock) store_cut<OUT>(row, v, a.dim, zero);
    }
  }
}

// ---------------------------------------------------------------------------
// All of it in one launch, for up to kOneSort tokens: block 0 sorts in LDS, by
// the same steps with 16 wavefronts (few tokens: several blocks, by counting), and
// the others meanwhile write the zeros.
// A block of those goes over all tokens for the rows of its own that are named.
// ---------------------------------------------------------------------------
constexpr uint32_t kOneSort = 16384, kOneThreads = 1024, kOneWaves = 16, kOneRounds = kOneSort / kOneThreads;
constexpr uint32_t kMapRows = 1u << 16;

struct OneArgs {
  const int64_t* tokens;
  uint32_t *keys, *at;  // sorted
  uint32_t n, vocab, bits, passes, sorters;  // sorters: the blocks that sort
  void* dtable;  // of the zeros
  uint64_t stride;
  uint32_t dim, vecs, shift;  // 1 << shift lanes to a row
};

// Few tokens: a block finds the places of 64 of them, 16 lanes to a token, by
// going over all keys (333 tokens: 3 us, where two passes of one block take 9).
constexpr uint32_t kCountTokens = 1024, kCountEach = 64;

__device__ __forceinline__ void sort_by_counting(const OneArgs& a, uint32_t* keys) {
  const uint32_t t = threadIdx.x;
  uint32_t key = 0xFFFFFFFFu;  // behind all others
  if (t < a.n) {
    const int64_t token = a.tokens[t];
    key = token >= 0 && token < (int64_t)a.vocab ? (uint32_t)token : a.vocab;
  }
  keys[t] = key;
  __syncthreads();
  const uint32_t i = blockIdx.x * kCountEach + t / 16;
  const uint32_t own = keys[min(i, kCountTokens - 1)];
  uint32_t place = 0;
  for (uint32_t j0 = t % 16 * 4; j0 < a.n; j0 += 64) {
    const u32x4 k = *reinterpret_cast<const u32x4*>(keys + j0);
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) place += (k[j] < own) | ((k[j] == own) & (j0 + j < i));
  }
  place += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)place, 0x128, 0xF, 0xF, false);  // row_ror:8, 4, 2, 1
  place += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)place, 0x124, 0xF, 0xF, false);
  place += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)place, 0x122, 0xF, 0xF, false);
  place += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)place, 0x121, 0xF, 0xF, false);
  if (t % 16 == 0 && i < a.n) {
    a.keys[place] = own;
    a.at[place] = i;
  }
}

__device__ __forceinline__ void sort_in_lds(const OneArgs& a, uint32_t* keys, uint16_t* at, uint16_t (*count)[kDigits],
                                            uint32_t* sums) {
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const uint32_t rounds = (a.n + kOneThreads - 1) / kOneThreads, begin = wave * rounds * 64 + lane;
  for (uint32_t pass = 0, done = 0; pass < a.passes; ++pass) {
    const uint32_t bits = (a.bits - done + a.passes - pass - 1) / (a.passes - pass), digits = 1u << bits;
    uint32_t key[kOneRounds], from[kOneRounds], rank[kOneRounds];
#pragma unroll
    for (uint32_t r = 0; r < kOneRounds; ++r) {
      const uint32_t i = begin + r * 64;
      key[r] = from[r] = 0;
      if (r < rounds && i < a.n) {
        if (pass == 0) {
          const int64_t token = a.tokens[i];
          key[r] = token >= 0 && token < (int64_t)a.vocab ? (uint32_t)token : a.vocab;
          from[r] = i;
        } else {
          key[r] = keys[i];
          from[r] = at[i];
        }
      }
    }
    for (uint32_t i = t; i < kOneWaves * kDigits / 2; i += kOneThreads) reinterpret_cast<uint32_t*>(count)[i] = 0;
    __syncthreads();
#pragma unroll
    for (uint32_t r = 0; r < kOneRounds; ++r) {
      if (r < rounds) {
        const bool has = begin + r * 64 < a.n;
        const uint32_t d = key[r] >> done & (digits - 1);
        uint64_t same = __ballot(has);
        for (uint32_t b = 0; b < bits; ++b) {
          const uint64_t one = __ballot(d >> b & 1);
          same &= (d >> b & 1) ? one : ~one;
        }
        const uint32_t before = __popcll(same & ((1ull << lane) - 1));
        const uint32_t seen = count[wave][d];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (has && before == 0) count[wave][d] = (uint16_t)(seen + __popcll(same));
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        rank[r] = seen + before;
      }
    }
    __syncthreads();
    // thread 2 d + h: digit d, wavefronts 8 h .. 8 h + 7
    const uint32_t d = t / 2, w0 = t % 2 * 8;
    uint32_t sum = 0;
#pragma unroll
    for (uint32_t w = 0; w < 8; ++w) sum += count[w0 + w][d];
    const uint32_t own = sum;
#pragma unroll
    for (uint32_t s = 1; s < 64; s <<= 1) {
      const uint32_t up = __shfl_up(sum, s, 64);
      if (lane >= s) sum += up;
    }
    if (lane == 63) sums[wave] = sum;
    __syncthreads();
    uint32_t to = sum - own;
    for (uint32_t w = 0; w < wave; ++w) to += sums[w];
#pragma unroll
    for (uint32_t w = 0; w < 8; ++w) {
      const uint32_t c = count[w0 + w][d];
      count[w0 + w][d] = (uint16_t)to;
      to += c;
    }
    __syncthreads();
    const bool last = pass + 1 == a.passes;
#pragma unroll
    for (uint32_t r = 0; r < kOneRounds; ++r) {
      if (r < rounds && begin + r * 64 < a.n) {
        const uint32_t p = count[wave][key[r] >> done & (digits - 1)] + rank[r];
        if (last) {
          a.keys[p] = key[r];
          a.at[p] = from[r];
        } else {
          keys[p] = key[r];
          at[p] = (uint16_t)from[r];
        }
      }
    }
    __syncthreads();
    done += bits;
  }
}

template <int OUT>
__global__ void __launch_bounds__(kOneThreads) one_sort_kernel(const OneArgs a) {
  typedef typename Vec<OUT>::T T;
  __shared__ __align__(16) uint32_t keys[kOneSort];
  __shared__ uint16_t at[kOneSort], count[kOneWaves][kDigits];
  __shared__ uint32_t sums[kOneWaves];
  if (blockIdx.x < a.sorters) {
    if (a.n <= kCountTokens) sort_by_counting(a, keys);
    else sort_in_lds(a, keys, at, count, sums);
    return;
  }
  // unit by unit in turn, a unit being the rows that the block writes at a time
  const uint32_t t = threadIdx.x, blocks = gridDim.x - a.sorters, b = blockIdx.x - a.sorters, lanes = 1u << a.shift;
  const uint32_t unit = kOneThreads >> a.shift, units = kMapRows / unit;
  uint32_t* named = keys;  // one bit to a row
  const float zero[Lane<OUT>::N] = {};
  const uint64_t all = ((uint64_t)a.vocab + unit - 1) / unit;
  for (uint64_t first = b; first < all; first += (uint64_t)blocks * units) {
    const uint32_t n = (uint32_t)min((all - first + blocks - 1) / blocks, (uint64_t)units);  // units of this round
    __syncthreads();
    for (uint32_t i = t; i < (n * unit + 31) / 32; i += kOneThreads) named[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (uint32_t i = t; i < a.n; i += kOneThreads) {
      const int64_t token = a.tokens[i];
      if (token < 0 || token >= (int64_t)a.vocab) continue;
      const uint32_t u = (uint32_t)token / unit, turn = u / blocks;
      if (u % blocks != b || u < first || (turn - (uint32_t)first / blocks) >= n) continue;
      const uint32_t bit = (turn - (uint32_t)first / blocks) * unit + (uint32_t)token % unit;
      atomicOr(&named[bit / 32], 1u << (bit % 32));
    }
    __syncthreads();
    for (uint32_t i = 0; i < n; ++i) {
      const uint32_t in = t >> a.shift, bit = i * unit + in;
      const uint64_t r = (first + (uint64_t)i * blocks) * unit + in;
      if (r >= a.vocab || (named[bit / 32] >> (bit % 32) & 1)) continue;
      T* row = static_cast<T*>(a.dtable) + r * a.stride;
      for (uint32_t v = t & (lanes - 1); v < a.vecs; v += lanes) store_cut<OUT>(row, v, a.dim, zero);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
constexpr uint32_t kMaxDim = 1u << 20;
constexpr uint64_t kMaxTokens = 1u << 28;  // of the gradient: a launch's threads fit 32 bits

uint64_t up256(uint64_t n) { return (n + 255) / 256 * 256; }

// Workspace: two copies of (keys, positions), the histogram, the partial sums.
struct Space {
  uint64_t keys[2], at[2], hist, totals, partial, bytes;
  uint32_t blocks, tile, tiles, row;  // row: floats of a partial row
};
Space space_of(uint64_t n, uint32_t dim) {
  Space s;
  s.blocks = (uint32_t)((n + kSortKeys - 1) / kSortKeys);
  s.tile = n <= kFewTokens ? kFewTile : kTile;
  s.tiles = (uint32_t)((n + s.tile - 1) / s.tile);
  s.row = (dim + 7) / 8 * 8;
  uint64_t at = 0;
  const auto take = [&](uint64_t bytes) {
    const uint64_t here = at;
    at += up256(bytes);
    return here;
  };
  for (int i = 0; i < 2; ++i) {
    s.keys[i] = take(n * 4);
    s.at[i] = take(n * 4);
  }
  s.hist = take((uint64_t)kDigits * s.blocks * 4);
  s.totals = take(kDigits * 4);
  // the most of any number of tokens up to n, of which 4096 have as many tiles as
  // 16,384: a workspace serves fewer tokens too
  const uint64_t few = (std::min<uint64_t>(n, kFewTokens) + kFewTile - 1) / kFewTile;
  s.partial = take(std::max<uint64_t>(s.tiles, few) * 2 * s.row * 4);
  s.bytes = std::max<uint64_t>(at, 256);
  return s;
}

int check_table(const void* table, int dtype, uint32_t vocab, uint32_t dim, uint64_t stride, const char* who) {
  if (!known_dtype(dtype)) return fail(ZERO_EINVAL, "%s: unknown dtype %d", who, dtype);
  if (vocab == 0 || vocab > (uint32_t)INT32_MAX) return fail(ZERO_EINVAL, "%s: vocab %u outside [1, 2^31)", who, vocab);
  if (dim == 0 || dim > kMaxDim) return fail(ZERO_EINVAL, "%s: dim %u outside [1, 2^20]", who, dim);
  if (stride < dim) return fail(ZERO_EINVAL, "%s: rows of %u elements overlap at a stride of %llu", who, dim,
                                (unsigned long long)stride);
  if (vocab > UINT64_MAX / 8 / stride) return fail(ZERO_EINVAL, "%s: vocab * stride overflows", who);
  if (!table || !multiple_of(table, dtype_bytes(dtype)))
    return fail(ZERO_EINVAL, "%s: the table is NULL or not aligned to its elements", who);
  return ZERO_OK;
}

}  // namespace
}  // namespace zs

using namespace zs;

extern "C" int zero_embedding(const void* table, int dtype, uint32_t vocab, uint32_t dim, uint64_t stride,
                              const int64_t* tokens, uint64_t n_tokens, double scale, void* out, hipStream_t stream) {
  static const char* who = "zero_embedding";
  clear_error();
  int rc = check_table(table, dtype, vocab, dim, stride, who);
  if (rc) return rc;
  if (!std::isfinite((float)scale)) return fail(ZERO_EINVAL, "%s: scale must be finite in fp32", who);
  if (n_tokens > UINT64_MAX / 8 / dim) return fail(ZERO_EINVAL, "%s: n_tokens * dim overflows", who);
  if (n_tokens == 0) return ZERO_OK;
  if (!tokens || !multiple_of(tokens, 8) || !out || !multiple_of(out, dtype_bytes(dtype)))
    return fail(ZERO_EINVAL, "%s: tokens or out is NULL or not aligned to its elements", who);
  if ((rc = begin_launch())) return rc;
  with_dtype(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    const uint32_t vecs = (dim + Lane<DT>::N - 1) / Lane<DT>::N;
    uint32_t shift = 0;
    while ((1u << shift) < vecs && (1u << shift) < (uint32_t)kBlock) ++shift;
    const EmbedArgs a = {table, tokens, out, n_tokens, stride, vocab, dim, vecs, (float)scale};
    const uint64_t rows = kBlock >> shift;
    const uint32_t grid = chunk_grid((n_tokens + rows - 1) / rows, 0);
    hipLaunchKernelGGL(embed_kernel<DT>, grid, kBlock, 0, stream, a, shift);
  });
  return launch_status(who);
}

extern "C" int zero_embedding_workspace_bytes(uint64_t n_tokens, uint32_t dim, uint64_t* bytes) {
  static const char* who = "zero_embedding_workspace_bytes";
  clear_error();
  if (!bytes) return fail(ZERO_EINVAL, "%s: bytes is NULL", who);
  if (dim == 0 || dim > kMaxDim) return fail(ZERO_EINVAL, "%s: dim %u outside [1, 2^20]", who, dim);
  if (n_tokens > kMaxTokens) return fail(ZERO_ERANGE, "%s: n_tokens beyond 2^28", who);
  *bytes = space_of(n_tokens, dim).bytes;
  return ZERO_OK;
}

extern "C" int zero_embedding_grad(const zero_embedding_grad_args* p, hipStream_t stream) {
  static const char* who = "zero_embedding_grad";
  clear_error();
  if (!p) return fail(ZERO_EINVAL, "%s: args is NULL", who);
  int rc = check_table(p->dtable, p->table_dtype, p->vocab, p->dim, p->stride, who);
  if (rc) return rc;
  if (!known_dtype(p->dtype)) return fail(ZERO_EINVAL, "%s: unknown dtype %d", who, p->dtype);
  if (p->table_dtype != p->dtype && p->table_dtype != ZERO_F32)
    return fail(ZERO_EINVAL, "%s: dtable must have the dtype of dout or fp32", who);
  if (!std::isfinite((float)p->scale)) return fail(ZERO_EINVAL, "%s: scale must be finite in fp32", who);
  if (p->n_tokens > kMaxTokens) return fail(ZERO_EINVAL, "%s: n_tokens beyond 2^28", who);
  const Space s = space_of(p->n_tokens, p->dim);
  if (p->n_tokens > 0) {
    if (!p->dout || !p->tokens || !multiple_of(p->dout, dtype_bytes(p->dtype)) || !multiple_of(p->tokens, 8))
      return fail(ZERO_EINVAL, "%s: dout or tokens is NULL or not aligned to its elements", who);
    if (!p->workspace) return fail(ZERO_EINVAL, "%s: workspace is NULL", who);
    if (p->workspace_bytes < s.bytes)
      return fail(ZERO_EINVAL, "%s: workspace needs %llu bytes, got %zu", who, (unsigned long long)s.bytes,
                  p->workspace_bytes);
    if (!multiple_of(p->workspace, 256)) return fail(ZERO_EINVAL, "%s: workspace must be 256-byte aligned", who);
  }
  if (p->n_tokens == 0 && p->accumulate) return ZERO_OK;
  if ((rc = begin_launch())) return rc;
  char* ws = static_cast<char*>(p->workspace);
  GradArgs g = {};
  g.dout = p->dout;
  g.dtable = p->dtable;
  g.stride = p->stride;
  g.n = (uint32_t)p->n_tokens;
  g.vocab = p->vocab;
  g.dim = p->dim;
  g.scale = (float)p->scale;
  g.accumulate = p->accumulate != 0;
  g.tile = s.tile;
  // Alone, one block's sort takes longer than several blocks' passes from some 10,000
  // tokens on (onto a gradient: 8192 tokens 58 us and 61, 16,384 tokens 115 and 103);
  // beside the zeros, which several passes have a launch of their own for, it is no
  // slower at any size (16,384 tokens of 128,000 x 4096 258 and 274, of 128,000 x 64 66
  // and 74, of 18,397 x 1 68 both ways; 8193 tokens of that 53 and 64).
  const bool one = g.n > 0 && g.n <= (g.accumulate ? kOneSort / 2 : kOneSort);
  if (g.n > 0) {
    // keys are 0 .. vocab: passes of equal width, 9 bits at most
    uint32_t bits = 1;
    while (bits < 32 && p->vocab >> bits) ++bits;
    const uint32_t passes = (bits + kMaxBits - 1) / kMaxBits;
    uint32_t* const keys[2] = {reinterpret_cast<uint32_t*>(ws + s.keys[0]), reinterpret_cast<uint32_t*>(ws + s.keys[1])};
    uint32_t* const at[2] = {reinterpret_cast<uint32_t*>(ws + s.at[0]), reinterpret_cast<uint32_t*>(ws + s.at[1])};
    if (one) {
      with_dtype(p->table_dtype, [&](auto dt) {
        constexpr int OUT = decltype(dt)::value;
        const uint32_t vecs = (p->dim + Lane<OUT>::N - 1) / Lane<OUT>::N;
        const uint32_t sorters = g.n <= kCountTokens ? (g.n + kCountEach - 1) / kCountEach : 1;
        OneArgs a = {p->tokens, keys[0], at[0], g.n, p->vocab, bits, passes, sorters, p->dtable, p->stride, p->dim, vecs, 0};
        while ((1u << a.shift) < vecs && a.shift < 6) ++a.shift;
        const uint32_t grid = g.accumulate ? a.sorters : 256;
        hipLaunchKernelGGL(one_sort_kernel<OUT>, grid, kOneThreads, 0, stream, a);
      });
      g.keys = keys[0];
      g.at = at[0];
    } else {
      SortArgs a = {p->tokens, nullptr, nullptr, nullptr, nullptr, reinterpret_cast<uint32_t*>(ws + s.hist),
                    reinterpret_cast<uint32_t*>(ws + s.totals), g.n, p->vocab, s.blocks, 0, 0};
      for (uint32_t i = 0, done = 0; i < passes; ++i) {
        a.shift = done;
        a.bits = (bits - done + passes - i - 1) / (passes - i);
        done += a.bits;
        a.keys_out = keys[i & 1];
        a.at_out = at[i & 1];
        hipLaunchKernelGGL(histogram_kernel, s.blocks, kBlock, 0, stream, a);
        if (s.blocks > kScanBlocks) hipLaunchKernelGGL(scan_kernel, 1u << a.bits, kBlock, 0, stream, a);
        hipLaunchKernelGGL(scatter_kernel, s.blocks, kBlock, 0, stream, a);
        a.tokens = nullptr;
        a.keys = a.keys_out;
        a.at = a.at_out;
      }
      g.keys = a.keys;
      g.at = a.at;
    }
    if ((rc = launch_status(who))) return rc;
    g.partial = reinterpret_cast<float*>(ws + s.partial);
  }
  if (!g.accumulate && !one) {
    const uint32_t grid = (uint32_t)std::min<uint64_t>((p->vocab + kFillRows - 1) / kFillRows, 1u << 20);
    with_dtype(p->table_dtype, [&](auto dt) {
      constexpr int OUT = decltype(dt)::value;
      const uint32_t vecs = (p->dim + Lane<OUT>::N - 1) / Lane<OUT>::N;
      hipLaunchKernelGGL(fill_kernel<OUT>, grid, kBlock, 0, stream, g, vecs);
    });
    if ((rc = launch_status(who))) return rc;
  }
  if (g.n == 0) return ZERO_OK;
  with_dtype(p->dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    g.vecs = (p->dim + Lane<DT>::N - 1) / Lane<DT>::N;
    const dim3 grid(s.tiles, std::min(65535u, (g.vecs + kBlock - 1) / kBlock));
    if (p->table_dtype == ZERO_F32 && DT != ZERO_F32) {
      hipLaunchKernelGGL((sum_kernel<DT, ZERO_F32>), grid, kBlock, 0, stream, g);
      hipLaunchKernelGGL((join_kernel<DT, ZERO_F32>), grid, kBlock, 0, stream, g);
    } else {
      hipLaunchKernelGGL((sum_kernel<DT, DT>), grid, kBlock, 0, stream, g);
      hipLaunchKernelGGL((join_kernel<DT, DT>), grid, kBlock, 0, stream, g);
    }
  });
  return launch_status(who);
}
