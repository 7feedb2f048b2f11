// token_filter.hip -- sampling from given logits under a request's limits
// (gfx950).
//
// Row x at temperature T, with w_i = 2^((x_i - max x) log2(e) / T): the tokens
// in the order of falling logits, ties by rising index, are cut to the first
// top_k, of those to the ones with w >= min_p, of those to the shortest
// prefix whose weight reaches top_p of theirs; the token is the first one, by
// index, at which the running weight of the kept ones exceeds u of their sum.
//
// The borders decide tokens, and a row has up to V of them, so weights are
// computed in 64 bits and, wherever sums of them are compared, summed as
// integers: a sum does not depend on its order, and atomics may form it.  Their
// unit is 2^-scale of the largest weight, as fine as 62 bits hold the row's sum
// (Choice::scale).
//
// Two launches.  The first reads the rows once, all of the device sharing
// them, and leaves the largest logit of every group of 128 columns (and the
// sum of its weights, for rows without top_k and min_p).  The second gives
// each row a workgroup, which needs the groups that can hold a kept token
// only: no token below the k-th largest of k groups' maxima is among the k
// largest, none below max + T ln(min_p) passes min_p, and those below
// (1 - top_p) / V of the sum together do not reach what top_p leaves out.  Up to
// 128 tokens that are left are placed without sorting, up to 2048 sorted; else
// each border is found by counts and sums over bins of the row, narrowed until
// the border's bin fits the list.
#include "device_common.h"
#include "token_filter.h"

namespace dspark {

namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kCap = 2048, kBins = 2048, kPer = kCap / kThreads;
constexpr int kFew = 128;      // keys that a workgroup places without sorting
constexpr int kParts = 1024, kPartBits = 11;  // parts of a row whose masses are kept, of at least 2^kPartBits columns
static_assert(kBins == kCap && kParts <= kCap, "bins and masses share memory, and a scan's steps");
constexpr int kVec = 8;
constexpr int kStepBits = 9;          // log2 of
constexpr int64_t kStep = 64 * kVec;  // the columns a wave takes at once
static_assert(kStep == 1 << kStepBits, "columns of a step");
constexpr uint32_t kNone = 0x007FFFFFu;     // code of -inf: what can be drawn lies above
constexpr uint32_t kInfCode = 0xFF800000u;  // code of +inf
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));  // rows start at any element

__device__ __forceinline__ float value_of(uint32_t code) {
  return __uint_as_float((code & 0x80000000u) ? code & 0x7FFFFFFFu : ~code);
}

// Eight logits of a row from column v on, as loaded; -inf past its end.
template <bool BF>
struct Raw {
  u32x4_t w[BF ? 1 : 2];
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (BF) return (e & 1) ? bf16_hi(w[0][e >> 1]) : bf16_lo(w[0][e >> 1]);
    else return __uint_as_float(w[e >> 2][e & 3]);
  }
};
template <bool BF>
__device__ __forceinline__ Raw<BF> load8(const void* row, int64_t v, int64_t V) {
  Raw<BF> r;
  if (v + kVec <= V) {
    const u32x4_any_t* const src = (const u32x4_any_t*)((const char*)row + v * (BF ? 2 : 4));
    r.w[0] = src[0];
    if constexpr (!BF) r.w[1] = src[1];
  } else {
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const bool in = v + e < V;
      if constexpr (BF) {
        const uint32_t b = in ? ((const uint16_t*)row)[v + e] : 0xFF80u;
        if (e & 1) r.w[0][e >> 1] |= b << 16;
        else r.w[0][e >> 1] = b;
      } else {
        r.w[e >> 2][e & 3] = in ? ((const uint32_t*)row)[v + e] : 0xFF800000u;
      }
    }
  }
  return r;
}
template <bool BF>
__device__ __forceinline__ float load1(const void* row, int64_t v) {
  return BF ? bf16_lo(((const uint16_t*)row)[v]) : ((const float*)row)[v];
}

// 2^(j / 32), j = 0 .. 31, in LDS: 64 banks hold one table, so that lanes that
// read different entries never meet in a bank.
constexpr int kTable = 32;
__device__ __forceinline__ void fill_table(double* table) {  // a barrier is the caller's
  if (threadIdx.x < kTable) {
    // a polynomial through the Chebyshev points of [-1/2, 1/2], 1 exactly at zero, good to 2^-50
    const double t = threadIdx.x * (1.0 / kTable), n = t > 0.5 ? 1.0 : 0.0, f = t - n;
    double y = 0x1.e5e9f548e5726p-28;
    y = __builtin_fma(y, f, 0x1.b6571de2f2351p-24);
    y = __builtin_fma(y, f, 0x1.62bfe46117445p-20);
    y = __builtin_fma(y, f, 0x1.ffcb76789860fp-17);
    y = __builtin_fma(y, f, 0x1.4309130378460p-13);
    y = __builtin_fma(y, f, 0x1.5d87fe908f88ap-10);
    y = __builtin_fma(y, f, 0x1.3b2ab6fba385fp-7);
    y = __builtin_fma(y, f, 0x1.c6b08d7044119p-5);
    y = __builtin_fma(y, f, 0x1.ebfbdff82c590p-3);
    y = __builtin_fma(y, f, 0x1.62e42fefa39f7p-1);
    table[threadIdx.x] = __builtin_fma(y, f, 1.0) * (1.0 + n);
  }
}
// 2^(scale + t / 32) for t <= 0, to 2^-50 (1 at zero exactly): the table at t's
// integer, and a polynomial through the Chebyshev points of [-1/2, 1/2] for what
// is left of it.  Half the 64-bit operations of a polynomial over a whole
// octave, and these bound the kernels; one degree less, good to 2^-42, takes 1% off
// 2048 fp32 rows of 151936 (734 to 726 us) and moves borders that can be told.
__device__ __forceinline__ double exp2_32nds(double t, int scale, const double* table) {
  t = __builtin_fmax(t, -64000.0);  // -inf too: 2^-2000 is zero
  const double k = t + 0x1.8p52;    // t's integer in the low bits
  const int n = (int)(uint32_t)__builtin_bit_cast(uint64_t, k);
  const double f = t - (k - 0x1.8p52);
  double y = 0x1.5d884e708e6aap-35;
  y = __builtin_fma(y, f, 0x1.3b2b1bee88b09p-27);
  y = __builtin_fma(y, f, 0x1.c6b08d70400d0p-20);
  y = __builtin_fma(y, f, 0x1.ebfbdff8131c3p-13);
  y = __builtin_fma(y, f, 0x1.62e42fefa39efp-6);
  return __builtin_ldexp(table[n & (kTable - 1)] * __builtin_fma(y, f, 1.0), (n >> 5) + scale);
}
// Weight of a logit relative to a number m that is not below it; kappa: 32 log2(e) / T.
__device__ __forceinline__ double weight64(float x, float m, double kappa, const double* table) {
  return exp2_32nds(((double)x - (double)m) * kappa, 0, table);
}

// The limits of a row as its kernels use them.
struct Limits {
  double kappa;  // 32 log2(e) / T
  double min_p;  // 0: off, at most 1
  float T;
  float top_p;
  int64_t k;     // V: off
  bool greedy, nucleus;
  bool full;     // every token can be kept: the sum over the row is needed
};
__device__ __forceinline__ Limits limits_of(const TokenLimits& l, int64_t b, int64_t V) {
  Limits r;
  r.T = l.temperature ? l.temperature[b] : l.all_temperature;
  const int64_t k = l.top_k ? l.top_k[b] : l.all_top_k;
  r.top_p = l.top_p ? l.top_p[b] : l.all_top_p;
  const float m = l.min_p ? l.min_p[b] : l.all_min_p;
  r.greedy = !(r.T >= 1e-5f);
  r.kappa = kTable * 1.4426950408889634 / (double)(r.greedy ? 1.0f : r.T);
  r.k = k > 0 && k < V ? k : V;
  r.nucleus = r.top_p < 1.0f;
  r.min_p = m > 0.0f ? __builtin_fmin((double)m, 1.0) : 0.0;
  r.full = !r.greedy && r.k == V && r.min_p == 0.0;
  return r;
}

// ---------------------------------------------------------------- sums of 64 bits
__device__ __forceinline__ uint64_t shfl_u64(uint64_t v, int lane) {
  return ((uint64_t)__shfl((uint32_t)(v >> 32), lane, 64) << 32) | __shfl((uint32_t)v, lane, 64);
}
template <typename T>
__device__ __forceinline__ T shift_up(T v, int by) {  // lane l - by's value
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint64_t s = ((uint64_t)__shfl_up((uint32_t)(u >> 32), by, 64) << 32) | __shfl_up((uint32_t)u, by, 64);
  return __builtin_bit_cast(T, s);
}
template <typename T>
__device__ __forceinline__ T wave_scan(T v) {  // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int by = 1; by < 64; by *= 2) {
    const T o = shift_up(v, by);
    if (lane >= by) v += o;
  }
  return v;
}
__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1)
    v += ((uint64_t)__shfl_xor((uint32_t)(v >> 32), off, 64) << 32) | __shfl_xor((uint32_t)v, off, 64);
  return v;
}

}  // namespace

// ---------------------------------------------------------------- groups
// A wave takes 512 columns of a row at a time, 16 lanes a group.  2048 fp32 rows
// of 151936 with their sums take 263 us (4.7 TB/s, the vector units 0.96 busy with
// 64-bit weights), 320 bf16 rows of 129280, a few with sums, 27 us, all 39, none
// 16, one row 4.6.
constexpr int kGroupThreads = 256, kTurns = 4;                          // turns of a wave
constexpr int kGroupSlice = kGroupThreads / 64 * kTurns * 64 * kVec;   // columns of a workgroup

template <bool BF>
__global__ __launch_bounds__(kGroupThreads) void filter_groups_kernel(FilterParams p, int64_t r0, unsigned slices) {
  const int64_t n = r0 + blockIdx.x / slices;
  const int lane = threadIdx.x & 63;
  const int64_t v0 = (int64_t)(blockIdx.x % slices) * kGroupSlice + (threadIdx.x >> 6) * (kTurns * 64 * kVec) + lane * kVec;
  const char* const row = (const char*)p.logits + n * p.V * (BF ? 2 : 4);
  const int64_t G = filter_groups(p.V);
  const Limits lim = limits_of(p.limits, n / p.M, p.V);
  __shared__ double table[kTable];
  Raw<BF> x[kTurns];
#pragma unroll
  for (int j = 0; j < kTurns; ++j) x[j] = load8<BF>(row, v0 + j * 64 * kVec, p.V);
  fill_table(table);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kTurns; ++j) {
    const int64_t v = v0 + j * 64 * kVec;
    float m = x[j][0];
    bool nan = false;  // which a maximum passes over
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      nan = nan || x[j][e] != x[j][e];
      m = __builtin_fmaxf(m, x[j][e]);
    }
    uint32_t top = nan ? 0xFFFFFFFFu : ordered_code(m);
#pragma unroll
    for (int off = 1; off < 16; off *= 2) top = max(top, (uint32_t)__shfl_xor(top, off, 64));
    if ((lane & 15) == 0 && v < p.V) p.tops[n * G + v / kFilterGroup] = top;
    if (lim.full) {
      double z = 0.0;
      if (top > kNone && top < kInfCode) {
        const float all = value_of(top);
#pragma unroll
        for (int e = 0; e < kVec; ++e) z += weight64(x[j][e], all, lim.kappa, table);
      }
#pragma unroll
      for (int off = 1; off < 16; off *= 2) z += __shfl_xor(z, off, 64);
      if ((lane & 15) == 0 && v < p.V) p.sums[n * G + v / kFilterGroup] = z;
    }
  }
}

// ---------------------------------------------------------------- choice
namespace {

struct Shared {
  uint64_t keys[kCap];
  union {
    uint64_t mass[kCap];                // of the sorted keys, or bins
    float stack[kWaves][63 + kStep];    // logits on their way to masses
  };
  uint64_t part[kParts];
  double table[kTable];
  uint64_t wave[kWaves];
  uint64_t lo, hi, found, before;
  uint32_t count;
  int at;
};

// Exclusive prefix of a value a thread, and the total.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* total, Shared& s) {
  const T up = wave_scan(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) s.wave[threadIdx.x >> 6] = __builtin_bit_cast(uint64_t, up);
  __syncthreads();
  T base = T(0), all = T(0);
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const T x = __builtin_bit_cast(T, s.wave[w]);
    if (w < (int)(threadIdx.x >> 6)) base += x;
    all += x;
  }
  *total = all;
  return base + (up - v);
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, Shared& s) {
  v = wave_max_u32_to_lane63(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) s.wave[threadIdx.x >> 6] = v;
  __syncthreads();
  uint64_t m = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) m = max_u64(m, s.wave[w]);
  return (uint32_t)m;
}

// Ascending sort of the list's n keys (a bitonic network).
__device__ __forceinline__ void sort_keys(Shared& s, int n) {
  int size = 2;
  while (size < n) size *= 2;
  __syncthreads();
  for (int i = n + threadIdx.x; i < size; i += kThreads) s.keys[i] = ~0ull;
  __syncthreads();
  for (int k = 2; k <= size; k *= 2)
    for (int j = k / 2; j > 0; j /= 2) {
      for (int i = threadIdx.x; i < size; i += kThreads) {
        const int o = i ^ j;
        if (o > i) {
          const uint64_t a = s.keys[i], b = s.keys[o];
          if ((a > b) == ((i & k) == 0)) {
            s.keys[i] = b;
            s.keys[o] = a;
          }
        }
      }
      __syncthreads();
    }
}

// A token's place in the falling order: rising keys.
__device__ __forceinline__ uint64_t order_key(uint32_t code, uint32_t i) { return ((uint64_t)~code << 32) | i; }
__device__ __forceinline__ uint32_t key_code(uint64_t k) { return ~(uint32_t)(k >> 32); }

// Rows of more columns than this take the WIDE form.  The scale of the other one
// goes by V weights of one, so that what a sum of kept weights, which is at
// least one, loses to its roundings is at most V 2^-(scale + 1): 2^-27 of it at
// this size, but 1/8 at V = 2^30, where a tail of a tenth of the row vanished.
// The scale of the WIDE form goes by the row: by its sum where that is known, by
// top_k up to this number, else by 128 times the sum of the largest weights of
// the groups that can hold a kept token.  A sum then loses at most V 2^-62 of
// itself by the first, 2^-26 by the second, 2^-25 by the third (as the kept
// weights sum to min(1, k / groups) of those largest ones or more).  Past 2^51
// the integers take a conversion of six instructions: one token of 129280 columns
// takes 17.7 us in this form, against 17.2, 2048 rows of 151936 730 against 726,
// and 16 flat rows of 2^20 2.95 ms against 2.84.
constexpr int64_t kNarrowColumns = 1 << 18;

// A row on its way to a token.
template <bool BF, bool WIDE>
struct Choice {
  const char* row;
  int64_t V;
  double kappa, min_p;  // min_p in units of masses
  float m;         // the largest logit
  uint32_t bound;  // code below which nothing is kept
  int scale;       // weights are integers of 2^-scale
  int part;        // a part's columns are 2^part, so that there are at most kParts
  const uint32_t* tops;
  Shared* s;

  // The mass of a token that passes min_p, else 0.
  __device__ __forceinline__ uint64_t mass(float x) const {
    const double w = exp2_32nds(((double)x - (double)m) * kappa, scale, s->table);
    if constexpr (WIDE) return w >= min_p ? (uint64_t)__builtin_rint(w) : 0;
    // at most 2^51: the sum's mantissa is the rounded integer
    return w >= min_p ? __builtin_bit_cast(uint64_t, w + 0x1p52) & 0xFFFFFFFFFFFFFull : 0;
  }
  __device__ __forceinline__ uint64_t mass_of(uint32_t code) const { return mass(value_of(code)); }

  // f(logits, first column) for eight columns a lane, 512 a wave, wherever one
  // of the wave's groups reaches the bound, and done(part) after the last of a
  // part.  The waves take turns by parts.  LOADS such steps are loaded before
  // the first is worked on: a row has few waves to hide its loads behind.  (What
  // rarely runs takes one at a time: f stands in the code LOADS times.)
  template <int LOADS, typename F, typename D>
  __device__ __forceinline__ void steps(F f, D done) const {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int shift = part - kStepBits;  // steps of a part
    const uint32_t n = (uint32_t)((V + kStep - 1) / kStep), parts = ((n - 1) >> shift) + 1;
    const uint32_t mine = wave < (int)parts ? ((parts - 1 - wave) / kWaves + 1) << shift : 0;
    const int64_t G = filter_groups(V);
    auto step = [&](uint32_t q) __attribute__((always_inline)) {
      return ((wave + (q >> shift) * kWaves) << shift) + (q & ((1u << shift) - 1));
    };
    uint32_t open = 0xFFFFFFFFu;  // the part that has been begun
    // 64 of the wave's steps at a time, a lane each, to see which of them count
    for (uint32_t q0 = 0; q0 < mine; q0 += 64) {
      const int64_t i = step(q0 + lane);
      uint32_t t = 0;
#pragma unroll
      for (int j = 0; j < kStep / kFilterGroup; ++j)
        if (q0 + lane < mine && i * (kStep / kFilterGroup) + j < G) t = max(t, tops[i * (kStep / kFilterGroup) + j]);
      uint64_t live = __ballot(t >= bound);
      while (live) {
        Raw<BF> x[LOADS];
        uint32_t at[LOADS];
        int have = 0;
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
          if (!live) continue;
          at[j] = step(q0 + (uint32_t)__builtin_ctzll(live));
          x[j] = load8<BF>(row, (int64_t)at[j] * kStep + lane * kVec, V);
          live &= live - 1;
          have = j + 1;
        }
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
          if (j >= have) continue;
          if (open != at[j] >> shift) {
            if (open != 0xFFFFFFFFu) done(open);
            open = at[j] >> shift;
          }
          f(x[j], (int64_t)at[j] * kStep + lane * kVec);
        }
      }
    }
    if (open != 0xFFFFFFFFu) done(open);
  }
  // f(code, column) for the row's tokens that may be kept.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const float least = value_of(bound);
    steps<1>(
        [&](const Raw<BF>& x, int64_t v) __attribute__((always_inline)) {
#pragma unroll
          for (int e = 0; e < kVec; ++e)
            if (x[e] >= least) f(ordered_code(x[e]), (uint32_t)(v + e));
        },
        [](uint32_t) {});
  }

  // The mass of a wave's tokens that belong to one part.  Those to be counted
  // are moved together first, so that no lane is idle while masses are computed:
  // a border usually keeps a few in a hundred of a row.
  struct Part {
    uint64_t sum = 0;
    uint32_t held = 0;  // on the wave's stack
  };
  template <typename F>
  __device__ __forceinline__ void count(Part& q, const Raw<BF>& x, F take) const {
    float* const stack = s->stack[threadIdx.x >> 6];
    const uint32_t lane = threadIdx.x & 63;
    uint32_t n = 0;
#pragma unroll
    for (int e = 0; e < kVec; ++e) n += take(e) ? 1u : 0u;
    if (__ballot(n != 0) == 0) return;
    const uint32_t upto = wave_inclusive_sum_u32(n);
    float* to = stack + q.held + (upto - n);
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      if (take(e)) *to++ = x[e];
    q.held += (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
    __builtin_amdgcn_wave_barrier();
    while (q.held >= 128) {
      q.held -= 128;
      const float y = stack[q.held + lane], z = stack[q.held + 64 + lane];
      q.sum += mass(y) + mass(z);
    }
    if (q.held >= 64) {
      q.held -= 64;
      q.sum += mass(stack[q.held + lane]);
    }
    __builtin_amdgcn_wave_barrier();
  }
  __device__ __forceinline__ void close(Part& q, uint32_t at) const {
    const uint32_t lane = threadIdx.x & 63;
    if (lane < q.held) q.sum += mass(s->stack[threadIdx.x >> 6][lane]);
    const uint64_t t = wave_sum_u64(q.sum);
    if (lane == 0) s->part[at] = t;
    q = Part{};
    __builtin_amdgcn_wave_barrier();
  }

  // Appends those of eight logits that take(e) names to the list.
  template <typename F>
  __device__ __forceinline__ void append(const Raw<BF>& x, int64_t v, F take) const {
    uint32_t n = 0;
#pragma unroll
    for (int e = 0; e < kVec; ++e) n += take(e) ? 1u : 0u;
    if (__ballot(n != 0) == 0) return;
    const uint32_t upto = wave_inclusive_sum_u32(n);
    uint32_t slot = 0;
    if ((threadIdx.x & 63) == 63) slot = atomicAdd(&s->count, upto);
    slot = (uint32_t)__builtin_amdgcn_readlane((int)slot, 63) + upto - n;
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      if (take(e)) {
        if (slot < kCap) s->keys[slot] = order_key(ordered_code(x[e]), (uint32_t)(v + e));
        ++slot;
      }
  }
  // The list of the tokens for which keep(code, key); returns how many there
  // are (more than kCap: the list is not whole), and their keys' range.
  template <typename F>
  __device__ __forceinline__ uint32_t gather(F keep, uint64_t* lo, uint64_t* hi) const {
    __syncthreads();
    if (threadIdx.x == 0) {
      s->count = 0;
      s->lo = ~0ull;
      s->hi = 0;
    }
    __syncthreads();
    uint64_t l = ~0ull, h = 0;
    each([&](uint32_t c, uint32_t i) {
      const uint64_t k = order_key(c, i);
      if (!keep(c, k)) return;
      l = k < l ? k : l;
      h = k > h ? k : h;
      const uint32_t at = atomicAdd(&s->count, 1u);
      if (at < kCap) s->keys[at] = k;
    });
    if (l <= h) {
      atomicMin((unsigned long long*)&s->lo, (unsigned long long)l);
      atomicMax((unsigned long long*)&s->hi, (unsigned long long)h);
    }
    __syncthreads();
    *lo = s->lo;
    *hi = s->hi;
    return s->count;
  }

  // The first of n amounts whose running sum, begun at `before`,
  // reaches the target: its place, and the sum before it.  One does.
  __device__ __forceinline__ int reach(const uint64_t* from, int n, uint64_t before, uint64_t target, uint64_t* sum) const {
    uint64_t a[kPer], t = 0, all;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = threadIdx.x * kPer + j;
      a[j] = i < n ? from[i] : 0;
      t += a[j];
    }
    uint64_t up = before + block_scan(t, &all, *s);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (up < target && target <= up + a[j]) {
        s->at = threadIdx.x * kPer + j;
        s->found = up;
      }
      up += a[j];
    }
    __syncthreads();
    *sum = s->found;
    return s->at;
  }
  __device__ __forceinline__ uint64_t total(const uint64_t* from, int n) const {
    uint64_t t = 0, all;
    __syncthreads();
    for (int i = threadIdx.x * kPer; i < threadIdx.x * kPer + kPer; ++i) t += i < n ? from[i] : 0;
    block_scan(t, &all, *s);
    return all;
  }

  // Even bins of a logit's distance from the largest, the last one for all
  // that lie further away.
  __device__ __forceinline__ float bins_of(float lowest) const {
    const float width = m - lowest;
    return width > 0.0f && width < 3.0e38f ? (float)kBins / width : 0.0f;
  }
  __device__ __forceinline__ int bin(uint32_t c, float per) const {
    return (int)fminf((m - value_of(c)) * per, (float)(kBins - 1));  // NaN (inf 0) falls into the last one
  }
  __device__ __forceinline__ void clear(uint64_t* p, int n) const {
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) p[i] = 0;
    __syncthreads();
  }
  template <bool MASS>
  __device__ __forceinline__ uint64_t amount(uint32_t c) const {
    if constexpr (MASS) return mass_of(c);
    else return 1;
  }

  // The key at which the running count (MASS: mass) of the n tokens with keys
  // in [lo, hi] reaches the target, begun at `before`: by bins of the key, of
  // a power of two each, until the border's bin fits the list.  The list may
  // hold them already.
  template <bool MASS>
  __device__ __forceinline__ uint64_t narrow(uint32_t n, uint64_t lo, uint64_t hi, uint64_t before, uint64_t target) const {
    while (n > kCap) {
      int shift = 0;
      while (((hi - lo) >> shift) >= kBins) ++shift;
      clear(s->mass, kBins);
      each([&](uint32_t c, uint32_t i) {
        const uint64_t k = order_key(c, i);
        if (k >= lo && k <= hi)
          atomicAdd((unsigned long long*)&s->mass[(k - lo) >> shift], (unsigned long long)amount<MASS>(c));
      });
      const uint64_t l = lo + ((uint64_t)reach(s->mass, kBins, before, target, &before) << shift);
      if (shift == 0) return l;
      const uint64_t h = l + ((1ull << shift) - 1);
      const uint64_t end = h < hi ? h : hi;
      n = gather([&](uint32_t, uint64_t k) { return k >= l && k <= end; }, &lo, &hi);
    }
    sort_keys(*s, (int)n);
    for (int i = threadIdx.x; i < (int)n; i += kThreads) s->mass[i] = amount<MASS>(key_code(s->keys[i]));
    uint64_t sum;
    return s->keys[reach(s->mass, (int)n, before, target, &sum)];
  }

  // The key of the k-th token; all of them if there are no more than k.
  __device__ __forceinline__ uint64_t border_count(uint64_t k, float lowest) const {
    const float per = bins_of(lowest);
    clear(s->mass, kBins);
    each([&](uint32_t c, uint32_t) { atomicAdd((uint32_t*)&s->mass[bin(c, per)], 1u); });
    if (k >= total(s->mass, kBins)) return ~0ull;
    uint64_t before, lo, hi;
    const int b = reach(s->mass, kBins, 0, k, &before);
    const uint32_t n = gather([&](uint32_t c, uint64_t) { return bin(c, per) == b; }, &lo, &hi);
    return narrow<false>(n, lo, hi, before, k);
  }

  // The key at which the mass of the tokens with keys up to `last` reaches that
  // share of `whole`, or of theirs where that is 0, the masses of the parts up
  // to there left in s->part.  Two passes: rough sums over even bins say which
  // bin the border lies in, then exact sums are formed of what lies above that
  // bin and its neighbours, whose tokens are sorted.  Should the border not lie
  // among them after all, or they not fit the list, it is searched for by exact
  // sums over bins.
  // CUT: not all tokens have keys up to `last`.
  template <bool CUT>
  __device__ __forceinline__ uint64_t border_mass(uint64_t last, float share, uint64_t whole, float lowest) const {
    constexpr int kLoads = CUT ? 1 : BF ? 4 : 2;
    const float per = bins_of(lowest), kf = (float)(kappa / kTable);
    const float least = value_of(bound);  // next to where min_p cuts, if it does
    auto within = [&](float x, int64_t i) __attribute__((always_inline)) {
      if constexpr (CUT) return order_key(ordered_code(x), (uint32_t)i) <= last;
      else return true;
    };
    // weights as integers of 2^-31 of a bound on their sum (float atomics on LDS
    // take twenty times as long as these)
    uint32_t* const bins = (uint32_t*)s->mass;
    int bits = 31;
    for (uint64_t z = whole ? (whole >> scale) + 1 : (uint64_t)V; z > 1; z = (z + 1) / 2) --bits;
    const float fb = (float)bits;
    clear(s->mass, kBins / 2);
    steps<kLoads>(
        [&](const Raw<BF>& x, int64_t v) __attribute__((always_inline)) {
          uint32_t w[kVec];
          int at[kVec];
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            const float d = m - x[e];
            w[e] = (uint32_t)(__builtin_amdgcn_exp2f(__builtin_fmaf(-d, kf, fb)) + 0.5f);
            at[e] = (int)fminf(d * per, (float)(kBins - 1));
          }
#pragma unroll
          for (int e = 0; e < kVec; ++e)
            if (x[e] >= least && within(x[e], v + e)) atomicAdd(&bins[at[e]], w[e]);
        },
        [](uint32_t) {});
    __syncthreads();
    double a[kPer], t = 0.0, all;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      a[j] = (double)bins[threadIdx.x * kPer + j];
      t += a[j];
    }
    double up = block_scan(t, &all, *s);
    const double goal = (double)share * (whole ? __builtin_ldexp((double)whole, bits - scale) : all);
    if (threadIdx.x == 0) s->at = kBins - 1;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (up < goal && goal <= up + a[j]) s->at = threadIdx.x * kPer + j;
      up += a[j];
    }
    __syncthreads();
    const int b0 = s->at - 1, b1 = s->at + 1;

    clear(s->part, kParts);
    if (threadIdx.x == 0) {
      s->count = 0;
      s->before = 0;
    }
    __syncthreads();
    uint64_t below = 0;
    Part over;
    const float high = b0 > 0 ? m - (float)b0 / per : __builtin_inff();
    const float low = b1 + 1 < kBins ? fmaxf(m - (float)(b1 + 1) / per, least) : least;
    steps<kLoads>(
        [&](const Raw<BF>& x, int64_t v) __attribute__((always_inline)) {
          count(over, x, [&](int e) __attribute__((always_inline)) { return x[e] > high && within(x[e], v + e); });
          append(x, v, [&](int e) __attribute__((always_inline)) {
            return x[e] >= low && !(x[e] > high) && within(x[e], v + e);
          });
          if (!whole) {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
              if (x[e] >= least && x[e] < low && within(x[e], v + e)) below += mass(x[e]);
          }
        },
        [&](uint32_t at) __attribute__((always_inline)) { close(over, at); });
    below = wave_sum_u64(below);
    if ((threadIdx.x & 63) == 0) atomicAdd((unsigned long long*)&s->before, (unsigned long long)below);
    __syncthreads();
    below = s->before;
    const uint32_t n = s->count;
    const uint64_t above = total(s->part, kParts);
    if (n <= kCap) {
      sort_keys(*s, (int)n);
      for (int i = threadIdx.x; i < (int)n; i += kThreads) s->mass[i] = mass_of(key_code(s->keys[i]));
      const uint64_t near = total(s->mass, (int)n), target = part_up(whole ? whole : above + near + below, share);
      if (above < target && target <= above + near) {
        uint64_t sum;
        const int at = reach(s->mass, (int)n, above, target, &sum);
        for (int i = threadIdx.x; i <= at; i += kThreads) {
          const int64_t v = (uint32_t)s->keys[i];
          atomicAdd((unsigned long long*)&s->part[v >> part], (unsigned long long)s->mass[i]);
        }
        const uint64_t key = s->keys[at];
        __syncthreads();
        return key;
      }
    }
    // by exact sums, from all that can be kept
    uint64_t l = ~0ull, h = 0, exact = 0;
    each([&](uint32_t c, uint32_t i) {
      const uint64_t k = order_key(c, i);
      if (k > last) return;
      l = k < l ? k : l;
      h = k > h ? k : h;
      exact += mass_of(c);
    });
    __syncthreads();
    if (threadIdx.x == 0) {
      s->lo = ~0ull;
      s->hi = 0;
      s->before = 0;
    }
    __syncthreads();
    atomicMin((unsigned long long*)&s->lo, (unsigned long long)l);
    atomicMax((unsigned long long*)&s->hi, (unsigned long long)h);
    atomicAdd((unsigned long long*)&s->before, (unsigned long long)exact);
    __syncthreads();
    l = s->lo;
    h = s->hi;
    exact = s->before;
    const uint64_t target = part_up(whole ? whole : exact, share);
    const uint64_t key = target > exact ? last : narrow<true>(kCap + 1, l, h, 0, target);
    parts_upto(key);
    return key;
  }

  // The masses of the parts, of the tokens with keys up to `last`.
  __device__ __forceinline__ void parts_upto(uint64_t last) const {
    const float least = value_of(bound);
    Part q;
    clear(s->part, kParts);
    steps<1>(
        [&](const Raw<BF>& x, int64_t v) __attribute__((always_inline)) {
          count(q, x, [&](int e) __attribute__((always_inline)) {
            return x[e] >= least && order_key(ordered_code(x[e]), (uint32_t)(v + e)) <= last;
          });
        },
        [&](uint32_t at) __attribute__((always_inline)) { close(q, at); });
    __syncthreads();
  }

  // ceil(share total), at least 1; floor(u total).
  static __device__ __forceinline__ uint64_t part_up(uint64_t total, float share) {
    const uint64_t f = share > 0.0f ? (uint64_t)((double)share * 0x1p40) : 0;
    const uint64_t up = __umul64hi(total, f << 24) + (total * (f << 24) != 0);
    return up > 0 ? up : 1;
  }
  static __device__ __forceinline__ uint64_t part_down(uint64_t total, float u) {
    const double c = fmin(fmax((double)u, 0.0), 1.0 - 0x1p-24);  // NaN: 0
    return __umul64hi(total, (uint64_t)(c * 0x1p40) << 24);
  }

  // The column at which the running mass, by index, of the tokens with keys up
  // to `last`, whose parts' masses stand in s->part, exceeds u of their sum,
  // which is left in *z.
  __device__ __forceinline__ int64_t draw(uint64_t last, float u, uint64_t* z) const {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    *z = total(s->part, kParts);
    uint64_t before, target = part_down(*z, u);
    int64_t a = (int64_t)reach(s->part, kParts, 0, target + 1, &before) << part;
    int64_t b = a + ((int64_t)1 << part) < V ? a + ((int64_t)1 << part) : V;
    target -= before;  // of what is left of it in [a, b)
    auto kept = [&](float x, int64_t i) __attribute__((always_inline)) -> uint64_t {
      const uint32_t c = ordered_code(x);
      return c >= bound && order_key(c, (uint32_t)i) <= last ? mass(x) : 0;
    };
    while (b - a > kStep) {
      const int64_t piece = ((b - a + kWaves - 1) / kWaves + kStep - 1) / kStep * kStep;
      const int64_t w0 = a + wave * piece, w1 = w0 + piece < b ? w0 + piece : b;
      uint64_t t = 0;
      for (int64_t v = w0 + lane * kVec; v < w1; v += kStep) {
        const Raw<BF> x = load8<BF>(row, v, V);
#pragma unroll
        for (int e = 0; e < kVec; ++e) t += kept(x[e], v + e);
      }
      t = wave_sum_u64(t);
      __syncthreads();
      if (lane == 0) s->wave[wave] = t;
      __syncthreads();
      uint64_t up = 0;
      int w = 0;
      while (w < kWaves - 1 && up + s->wave[w] <= target) up += s->wave[w++];
      target -= up;
      a += w * piece;
      b = a + piece < b ? a + piece : b;
    }
    // at most 512 columns, eight a lane: every wave finds the same
    uint64_t k[kVec], t = 0;
    const int64_t v = a + lane * kVec;
    const Raw<BF> x = load8<BF>(row, v < b ? v : V, V);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      k[e] = kept(x[e], v + e);
      t += k[e];
    }
    uint64_t run = wave_scan(t) - t;
    int64_t at = -1;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      if (at < 0 && run <= target && target < run + k[e]) at = v + e;
      run += k[e];
    }
    const uint64_t hit = __ballot(at >= 0);
    return (int64_t)shfl_u64((uint64_t)at, hit ? __builtin_ctzll(hit) : 0);
  }
};

}  // namespace

// A workgroup a row, two a CU (at 1024 threads 256 x 8 rows took 873 us instead of
// 740).  Nucleus rows of 151936 fp32 logits with tens of thousands of kept tokens
// take two more passes over themselves: 2048 of them 500 us, 2.37 GB at 4.7 TB/s;
// a row alone 69 us (62 at 1024 threads), 97 of 129280 standard normal logits in
// bf16, all barriers and loads that wait for each other.  With at most 128
// candidates a row takes 12 us.
template <bool BF, bool WIDE>
__global__ __launch_bounds__(kThreads, 4) void filter_choose_kernel(FilterParams p, int64_t r0) {
  __shared__ Shared s;
  fill_table(s.table);
  const int64_t n = r0 + blockIdx.x, V = p.V, G = filter_groups(V);
  const int tid = threadIdx.x, lane = tid & 63;
  const uint32_t* const tops = p.tops + n * G;
  const double* const sums = p.sums + n * G;
  const Limits lim = limits_of(p.limits, n / p.M, V);
  const float u = p.uniforms[n];
  Choice<BF, WIDE> c;
  c.row = (const char*)p.logits + n * V * (BF ? 2 : 4);
  c.V = V;
  c.kappa = lim.kappa;
  c.s = &s;
  auto scale_to = [&](int scale) __attribute__((always_inline)) {
    c.scale = scale;
    c.min_p = __builtin_ldexp(lim.min_p, scale);
  };
  // the scale at which a sum of weights below z, at least 1, is an integer below 2^62
  auto scale_by = [&](double z) __attribute__((always_inline)) {
    scale_to(62 - ((int)(__builtin_bit_cast(uint64_t, z) >> 52) - 1022));
  };
  if constexpr (!WIDE) {
    int bits = 0;
    while (((int64_t)1 << bits) < V) ++bits;
    scale_to(62 - bits < 51 ? 62 - bits : 51);
  }
  c.part = kPartBits;
  while (((V - 1) >> c.part) >= kParts) ++c.part;
  c.tops = tops;
  // a thread's groups are consecutive
  const int64_t per = (G + kThreads - 1) / kThreads, g0 = tid * per, g1 = g0 + per < G ? g0 + per : G;
  uint32_t own = 0, low = 0xFFFFFFFFu;
  for (int64_t g = g0; g < g1; ++g) {
    const uint32_t t = tops[g];
    own = max(own, t);
    if (t > kNone) low = min(low, t);
  }
  const uint32_t top = block_max(own, s);
  int64_t token = -1;
  float prob = 0.0f;
  auto finish = [&]() __attribute__((always_inline)) {
    if (tid == 0) {
      p.tokens[n] = token;
      p.probs[n] = prob;
    }
  };
  if (top <= kNone) return finish();  // nothing to draw from
  if (lim.greedy || top >= kInfCode) {
    // the first of the largest, in the first group that has it
    int64_t g = g0;
    while (g < g1 && tops[g] != top) ++g;
    const uint32_t not_mine = g < g1 ? 0xFFFFFFFFu - (uint32_t)g : 0u;
    g = 0xFFFFFFFFu - block_max(not_mine, s);
    uint32_t best = 0;
    for (int j = 0; j < kFilterGroup / 64; ++j) {
      const int64_t v = g * kFilterGroup + j * 64 + lane;
      if (v < V && ordered_code(load1<BF>(c.row, v)) == top) best = max(best, 0xFFFFFFFFu - (uint32_t)v);
    }
    best = (uint32_t)__builtin_amdgcn_readlane((int)wave_max_u32_to_lane63(best), 63);
    token = 0xFFFFFFFFu - best;
    prob = top == 0xFFFFFFFFu ? __builtin_nanf("") : 1.0f;
    return finish();
  }
  const float m = value_of(top);
  c.m = m;

  if (lim.full && !lim.nucleus) {
    // every token is kept: to the group by the groups' sums, then within it
    double t = 0.0, z;
    for (int64_t g = g0; g < g1; ++g)
      if (tops[g] > kNone) t += sums[g] * weight64(value_of(tops[g]), m, c.kappa, s.table);
    const double up = block_scan(t, &z, s), target = fmin(fmax((double)u, 0.0), 1.0 - 0x1p-24) * z;
    __syncthreads();
    if (tid == 0) s.found = 0;
    __syncthreads();
    // the last thread that begins at or below the target and holds anything
    if (t > 0.0 && up <= target) atomicMax((unsigned long long*)&s.found, (unsigned long long)tid + 1);
    __syncthreads();
    if (s.found == (uint64_t)tid + 1) {
      double run = up, begin = up;
      int64_t at = g0;
      for (int64_t g = g0; g < g1 && run <= target; ++g) {
        const double z = tops[g] > kNone ? sums[g] * weight64(value_of(tops[g]), m, c.kappa, s.table) : 0.0;
        if (z == 0.0) continue;
        at = g;
        begin = run;
        run += z;
      }
      s.lo = (uint64_t)at;
      s.hi = __builtin_bit_cast(uint64_t, begin);
    }
    __syncthreads();
    const int64_t v = (int64_t)s.lo * kFilterGroup + 2 * lane;
    double w[2];
    for (int e = 0; e < 2; ++e) {
      const float x = v + e < V ? load1<BF>(c.row, v + e) : -__builtin_inff();
      w[e] = weight64(x, m, c.kappa, s.table);
    }
    // the last token that begins at or below the target and weighs anything
    const double b0 = __builtin_bit_cast(double, s.hi) + (wave_scan(w[0] + w[1]) - (w[0] + w[1])), b1 = b0 + w[0];
    uint32_t best = 0;
    if (w[0] > 0.0 && b0 <= target) best = 2 * lane + 1;
    if (w[1] > 0.0 && b1 <= target) best = 2 * lane + 2;
    best = (uint32_t)__builtin_amdgcn_readlane((int)wave_max_u32_to_lane63(best), 63);
    token = (int64_t)s.lo * kFilterGroup + (best > 0 ? best - 1 : 0);
    if (best == 0) {  // rounding of the group's sum put the target before its first token
      const uint64_t some = __ballot(w[0] > 0.0 || w[1] > 0.0);
      const int l = some ? __builtin_ctzll(some) : 0;
      token = (int64_t)s.lo * kFilterGroup + 2 * l + (__shfl(w[0] > 0.0 ? 1 : 0, l, 64) ? 0 : 1);
    }
    prob = (float)(weight64(load1<BF>(c.row, token), m, c.kappa, s.table) / z);
    return finish();
  }

  // ---- a bound below which nothing is kept
  uint32_t bound = kNone + 1;
  if (lim.k <= kThreads) {
    // the k-th largest of the threads' maxima, to its upper 16 bits
    __syncthreads();
    s.keys[tid] = own;
    __syncthreads();
    uint32_t v[kWaves], kth = 0;
    for (int j = 0; j < kWaves; ++j) v[j] = (uint32_t)s.keys[j * 64 + lane];
    for (int bit = 31; bit >= 16; --bit) {
      const uint32_t t = kth | (1u << bit);
      int64_t cnt = 0;
      for (int j = 0; j < kWaves; ++j) cnt += __popcll(__ballot(v[j] >= t));
      if (cnt >= lim.k) kth = t;
    }
    bound = max(bound, kth);
  }
  if (lim.min_p > 0.0) {
    // a little below the border: the tokens next to it are looked at one by one
    const double x = (double)m + log(lim.min_p) * (double)lim.T;
    const float f = (float)(x - 1e-5 * (fabs(x) + fabs((double)m)));
    if (f > -3.0e38f) bound = max(bound, ordered_code(f));
  }
  uint64_t whole = 0;  // mass of the row where groups below the bound count too
  if (lim.full) {
    double t = 0.0, z;
    for (int64_t g = g0; g < g1; ++g)
      if (tops[g] > kNone) t += sums[g] * weight64(value_of(tops[g]), m, c.kappa, s.table);
    block_scan(t, &z, s);
    if constexpr (WIDE) scale_by(z);
    whole = (uint64_t)__builtin_rint(__builtin_ldexp(z, c.scale));
    // what weighs less than (1 - top_p) z / V reaches no more than 1 - top_p of
    // z with all its like (and a little less, for the roundings)
    const double share = (1.0 - fmax((double)lim.top_p, 0.0)) * 0.999, x = (double)m + log(share * z / (double)V) * (double)lim.T;
    const float f = (float)(x - 1e-5 * (fabs(x) + fabs((double)m)));
    if (f > -3.0e38f) bound = max(bound, min(ordered_code(f), top));
  }
  c.bound = min(bound, top);
  if constexpr (WIDE) {
    if (!lim.full && lim.k <= kNarrowColumns) {
      scale_by((double)lim.k);
    } else if (!lim.full) {
      double t = 0.0, z;
      for (int64_t g = g0; g < g1; ++g)
        if (tops[g] >= c.bound) t += weight64(value_of(tops[g]), m, c.kappa, s.table);
      block_scan(t, &z, s);
      scale_by(kFilterGroup * z);
    }
  }

  // ---- the groups that reach it, and their tokens, while they fit the list
  uint32_t mine = 0;
  for (int64_t g = g0; g < g1; ++g) mine += tops[g] >= c.bound;
  uint64_t groups;
  const uint64_t before = block_scan((uint64_t)mine, &groups, s);
  uint32_t count = kCap + 1;
  if (groups <= kCap) {
    uint32_t* const list = (uint32_t*)s.mass;
    uint32_t at = (uint32_t)before;
    __syncthreads();
    for (int64_t g = g0; g < g1; ++g)
      if (tops[g] >= c.bound) list[at++] = (uint32_t)g;
    if (tid == 0) s.count = 0;
    __syncthreads();
    constexpr uint32_t kTurn = kThreads / 16;  // 16 lanes a group
    const float least = value_of(c.bound);
    for (uint32_t i = (tid >> 6) * 4 + (lane >> 4), i0 = (tid >> 6) * 4; i0 < (uint32_t)groups; i += 4 * kTurn, i0 += 4 * kTurn) {
      if (__builtin_amdgcn_readfirstlane((int)__atomic_load_n(&s.count, __ATOMIC_RELAXED)) > kCap) break;  // it does not
      Raw<BF> x[4];
      int64_t v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t g = i + j * kTurn;
        v[j] = g < (uint32_t)groups ? (int64_t)list[g] * kFilterGroup + (tid & 15) * kVec : V;
        x[j] = load8<BF>(c.row, v[j], V);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c.append(x[j], v[j], [&](int e) __attribute__((always_inline)) { return x[j][e] >= least; });
    }
    __syncthreads();
    count = s.count;
  }
  uint64_t z;
  if (count <= kFew) {
    // Few tokens, as a top_k leaves: every wave holds all of them, two a lane, and
    // compares each with sixteen; the waves' counts and sums meet in LDS.  Four
    // barriers in place of two sorts and five scans.
    const int wave = tid >> 6;
    uint64_t* const places = s.mass;
    uint64_t* const befores = s.mass + kFew;
    uint64_t* const uptos = s.mass + 2 * kFew;
    uint64_t* const sums2 = s.mass + 3 * kFew;
    uint64_t key[2], w[2], n1[2] = {0, 0}, n2[2] = {0, 0}, n3[2] = {0, 0}, all = 0;
    if (tid < 3 * kFew + 2) s.mass[tid] = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      key[h] = lane + 64 * h < (int)count ? s.keys[lane + 64 * h] : ~0ull;
      w[h] = lane + 64 * h < (int)count ? c.mass_of(key_code(key[h])) : 0;
    }
    auto of = [&](const uint64_t (&v)[2], int j) __attribute__((always_inline)) {  // token 16 wave + j's
      const uint64_t x = wave < 4 ? v[0] : v[1];
      const int l = 16 * (wave & 3) + j;
      return ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), l) << 32) |
             (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, l);
    };
    auto meet = [&](uint64_t* to, uint64_t x) __attribute__((always_inline)) {
      atomicAdd((unsigned long long*)to, (unsigned long long)x);
    };
    __syncthreads();
    for (int j = 0; j < kFew / kWaves; ++j) {
      const uint64_t o = of(key, j);
#pragma unroll
      for (int h = 0; h < 2; ++h) n1[h] += o < key[h] ? 1 : 0;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) meet(&places[lane + 64 * h], n1[h]);
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) w[h] = places[lane + 64 * h] < (uint64_t)lim.k ? w[h] : 0;
    if (lim.nucleus) {
      for (int j = 0; j < kFew / kWaves; ++j) {
        const uint64_t o = of(key, j), x = of(w, j);
        all += x;
#pragma unroll
        for (int h = 0; h < 2; ++h) n2[h] += o < key[h] ? x : 0;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) meet(&befores[lane + 64 * h], n2[h]);
      if (lane == 0) meet(&sums2[0], all);
      __syncthreads();
      const uint64_t target = Choice<BF, WIDE>::part_up(whole ? whole : sums2[0], lim.top_p);
#pragma unroll
      for (int h = 0; h < 2; ++h) w[h] = befores[lane + 64 * h] < target ? w[h] : 0;
    }
    all = 0;
    for (int j = 0; j < kFew / kWaves; ++j) {
      const uint64_t o = of(key, j), x = of(w, j);
      all += x;
#pragma unroll
      for (int h = 0; h < 2; ++h) n3[h] += (uint32_t)o <= (uint32_t)key[h] ? x : 0;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) meet(&uptos[lane + 64 * h], n3[h]);
    if (lane == 0) meet(&sums2[1], all);
    __syncthreads();
    z = sums2[1];
    const uint64_t target = Choice<BF, WIDE>::part_down(z, u);
    token = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint64_t upto = uptos[lane + 64 * h];
      const uint64_t hit = __ballot(upto > target && upto - w[h] <= target);  // w is not zero then
      if (hit) token = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)key[h], __builtin_ctzll(hit));
    }
  } else if (count <= kCap) {
    sort_keys(s, (int)count);
    int kept = lim.k < (int64_t)count ? (int)lim.k : (int)count;
    for (int i = tid; i < kept; i += kThreads) s.mass[i] = c.mass_of(key_code(s.keys[i]));
    if (lim.nucleus) {
      uint64_t sum;
      const uint64_t all = c.total(s.mass, kept), target = Choice<BF, WIDE>::part_up(whole ? whole : all, lim.top_p);
      if (target <= all) kept = c.reach(s.mass, kept, 0, target, &sum) + 1;
    }
    z = c.total(s.mass, kept);
    const uint64_t target = Choice<BF, WIDE>::part_down(z, u);
    // by index: the key's halves change places, the lower one now the place in the list
    __syncthreads();
    uint64_t k[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid + j * kThreads;
      k[j] = i < kept ? (s.keys[i] << 32) | (uint32_t)i : 0;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (tid + j * kThreads < kept) s.keys[tid + j * kThreads] = k[j];
    sort_keys(s, kept);
    uint64_t a[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid + j * kThreads;
      a[j] = i < kept ? s.mass[(uint32_t)s.keys[i]] : 0;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (tid + j * kThreads < kept) s.mass[tid + j * kThreads] = a[j];
    uint64_t sum;
    token = (int64_t)(s.keys[c.reach(s.mass, kept, 0, target + 1, &sum)] >> 32);
  } else {
    // where the bins end: at the bound, or well below the groups' least maximum
    const float least = value_of(0xFFFFFFFFu - block_max(0xFFFFFFFFu - low, s));
    const float lowest = c.bound > kNone + 1 ? value_of(c.bound) : m - 4.0f * (m - least);
    uint64_t last = ~0ull;
    if (lim.k < V) last = c.border_count((uint64_t)lim.k, lowest);
    if (lim.nucleus && last != ~0ull) last = c.template border_mass<true>(last, lim.top_p, whole, lowest);
    else if (lim.nucleus) last = c.template border_mass<false>(last, lim.top_p, whole, lowest);
    else c.parts_upto(last);
    token = c.draw(last, u, &z);
  }
  prob = (float)(weight64(load1<BF>(c.row, token), m, c.kappa, s.table) / __builtin_ldexp((double)z, -c.scale));
  finish();
}

namespace {
// launch(r0, rows) for parts of the rows whose workgroups of `threads` fit one launch.
template <typename F>
hipError_t by_rows(int64_t rows, int64_t groups, int threads, F launch) {
  const int64_t step = kLaunchGroups / (threads / 256) / groups;
  if (step < 1) return hipErrorNotSupported;
  for (int64_t r = 0; r < rows; r += step) {
    launch(r, rows - r < step ? rows - r : step);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <bool BF>
hipError_t filter_go(const FilterParams& p, hipStream_t s) {
  const int64_t slices = (p.V + kGroupSlice - 1) / kGroupSlice;
  const hipError_t e = by_rows(p.rows, slices, kGroupThreads, [&](int64_t r, int64_t rows) {
    hipLaunchKernelGGL(filter_groups_kernel<BF>, dim3((unsigned)(rows * slices)), dim3(kGroupThreads), 0, s, p, r,
                       (unsigned)slices);
  });
  if (e != hipSuccess) return e;
  return by_rows(p.rows, 1, kThreads, [&](int64_t r, int64_t rows) {
    if (p.V > kNarrowColumns)
      hipLaunchKernelGGL((filter_choose_kernel<BF, true>), dim3((unsigned)rows), dim3(kThreads), 0, s, p, r);
    else
      hipLaunchKernelGGL((filter_choose_kernel<BF, false>), dim3((unsigned)rows), dim3(kThreads), 0, s, p, r);
  });
}
}  // namespace

hipError_t launch_token_filter(const FilterParams& p, bool bf16, hipStream_t s) {
  return bf16 ? filter_go<true>(p, s) : filter_go<false>(p, s);
}

}  // namespace dspark
