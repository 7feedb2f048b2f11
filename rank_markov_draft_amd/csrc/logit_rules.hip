// logit_rules.hip -- penalties for repeated tokens, biases and grammar masks
// on logits (gfx950).
//
// For row (b, k) and column v, with c the times v stands among the outputs
// counted for the row and "seen" whether it stands anywhere in the counted
// tokens (prompt or outputs):
//     x = logits[b, k, v]
//     seen:   x = x > 0 ? x / repetition[b] : x * repetition[b]
//     c > 0:  x = x - (frequency[b] * c + presence[b])
//     x = x + bias[b, v]
//     masked: x = -inf
// in fp32, rounded once to the logits' dtype.  A masked column is -inf
// whatever stood there, NaN included.
//
// The rules move every logit once and do next to no arithmetic, so they are
// bound by HBM; what could cost more than that is looking up, for every
// column, whether its token stands in the history.  A workgroup owns one
// request and one tile of the vocabulary: it walks the request's ids once,
// keeps those of its tile as a bitmap and counts in LDS, then streams the
// tile of the request's positions past that table.  The ids are re-read once
// per tile of the vocabulary, from L2; nothing is sorted or written to memory.
// 256 x 8 rows of 151936 in fp32, 2048 ids, all rules: 512 us, 5.0 TB/s; the
// gradient of 64 x 5 rows of 129280 in bf16, 1024 ids: 45 us (29 us without
// ids: a hit's logits are a line of their own).
#include "device_common.h"
#include "logit_rules.h"
#include "logit_rules_device.h"

namespace dspark {

namespace {

constexpr int kRuleThreads = 256;

// Adds the ids of request b that lie in [t0, t0 + tn) to a tile's table:
// every counted id to the bitmap, those past the prompt to the counts (null:
// not kept).  Lengths are clamped to the row, ids outside the vocabulary
// ignored.
__device__ __forceinline__ void count_history(const RuleSet& r, int64_t b, int64_t t0, int tn, uint32_t* seen,
                                              uint32_t* counts) {
  if (r.history == nullptr) return;
  int64_t len = r.lengths ? r.lengths[b] : r.history_len;
  len = len < 0 ? 0 : len > r.history_len ? r.history_len : len;
  int64_t prompt = r.prompt_lengths ? r.prompt_lengths[b] : 0;
  const int64_t* ids = r.history + b * r.history_stride;
  constexpr int U = 8;  // ids in flight per thread
  for (int64_t i0 = threadIdx.x; i0 < len; i0 += U * kRuleThreads) {
    int64_t id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u * kRuleThreads;
      id[u] = i < len ? ids[i] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint64_t c = (uint64_t)id[u] - (uint64_t)t0;
      if (id[u] >= 0 && c < (uint64_t)tn) {
        atomicOr(&seen[c >> 5], 1u << (c & 31));
        if (counts && i0 + u * kRuleThreads >= prompt) atomicAdd(&counts[c], 1u);
      }
    }
  }
}

// Vectors of rows that start at any element (an odd vocabulary): the hardware
// loads and stores 16 bytes at any address.
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));

// 8 consecutive values of a row as they are stored.
template <bool BF>
struct Raw8 {
  u32x4_t w[BF ? 1 : 2];
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (BF) {
      const uint32_t q = w[0][i >> 1];
      return (i & 1) ? bf16_hi(q) : bf16_lo(q);
    } else {
      return __uint_as_float(w[i >> 2][i & 3]);
    }
  }
};

// The first n of them (n < 8 at the row's end; the others are zero).
template <bool BF, bool STREAM>
__device__ __forceinline__ Raw8<BF> load8(const void* at, int n) {
  Raw8<BF> r;
#pragma unroll
  for (int h = 0; h < (BF ? 1 : 2); ++h) r.w[h] = u32x4_t{0u, 0u, 0u, 0u};
  if (n >= 8) {
#pragma unroll
    for (int h = 0; h < (BF ? 1 : 2); ++h) {
      const u32x4_any_t* const p = (const u32x4_any_t*)at + h;
      r.w[h] = STREAM ? __builtin_nontemporal_load(p) : *p;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if constexpr (BF) r.w[0][i >> 1] |= (uint32_t)((const uint16_t*)at)[i] << (16 * (i & 1));
        else r.w[i >> 2][i & 3] = ((const uint32_t*)at)[i];
      }
  }
  return r;
}
template <bool BF>
__device__ __forceinline__ void store8(void* at, int n, const float (&x)[8]) {
  u32x4_t w[2];
  if constexpr (BF) {
    w[0] = u32x4_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[h] = u32x4_t{__float_as_uint(x[4 * h]), __float_as_uint(x[4 * h + 1]), __float_as_uint(x[4 * h + 2]),
                     __float_as_uint(x[4 * h + 3])};
  }
  if (n >= 8) {
#pragma unroll
    for (int h = 0; h < (BF ? 1 : 2); ++h) __builtin_nontemporal_store(w[h], (u32x4_any_t*)at + h);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if constexpr (BF) ((uint16_t*)at)[i] = (uint16_t)(w[0][i >> 1] >> (16 * (i & 1)));
        else ((uint32_t*)at)[i] = w[i >> 2][i & 3];
      }
  }
}

// Biases of columns i .. i + N - 1 of the bias tensor (N 8 or 4; the first n exist).
template <int N>
__device__ __forceinline__ void bias8(const RuleSet& r, int64_t i, int n, float (&x)[8]) {
  if (n >= N) {
    if (r.bias_bf16) {
      typedef uint32_t words_t __attribute__((ext_vector_type(N / 2), aligned(2)));
      const words_t w = *(const words_t*)((const uint16_t*)r.bias + i);
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
    } else {
#pragma unroll
      for (int h = 0; h < N / 4; ++h) {
        const u32x4_t w = *(const u32x4_any_t*)((const float*)r.bias + i + 4 * h);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * h + e] = __uint_as_float(w[e]);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      x[e] = e >= n ? 0.0f : r.bias_bf16 ? bf16_lo(((const uint16_t*)r.bias)[i + e]) : ((const float*)r.bias)[i + e];
  }
}

}  // namespace

// A workgroup: T columns of one request, a span of its positions in groups of
// R, a thread 8 columns of a group's rows (and U such columns) at a time, so that
// R * U vectors are in flight while the bias and the table's bits of a column
// are read once for its R rows.
//
// The block's own tokens differ from row to row.  Before a group, those up to
// its first row join the table for good; the few within it only set their
// bit in `any`, and a column whose bit is set looks them up one by one.
template <bool BF, bool BWD, int R, int U>
__global__ __launch_bounds__(kRuleThreads) void logit_rules_kernel(RulesParams p, int T, int tiles, int64_t span,
                                                                   bool track, bool keep_counts) {
  extern __shared__ uint32_t rule_lds[];
  uint32_t* const any = rule_lds;                                        // T / 32 words
  uint32_t* const seen = rule_lds + T / 32;                              // T / 32 words
  uint32_t* const counts = keep_counts ? rule_lds + T / 16 : nullptr;    // T words
  __shared__ uint32_t blk[R];  // columns of the group's tokens k0 + 1 .. k0 + R - 1 relative to the tile, at 1 .. R - 1
  // request, and positions kb .. ke - 1 of it (spans of a multiple of R)
  const unsigned spans = (unsigned)((p.M + span - 1) / span), which = blockIdx.x / (unsigned)tiles;
  const int64_t b = which / spans;
  const int64_t kb = (int64_t)(which % spans) * span, ke = p.M - kb < span ? p.M : kb + span;
  const int64_t t0 = (int64_t)(blockIdx.x % (unsigned)tiles) * T;
  const int tn = (int)(p.V - t0 < T ? p.V - t0 : T);
  const int tid = threadIdx.x;
  constexpr int ES = BF ? 2 : 4;
  const Penalty pen = penalty_of(p.r, b);
  const int64_t* const ids = track && p.token_ids ? p.token_ids + b * p.M : nullptr;
  // the values and mask bits of a group's columns c0 (+ U - 1 strides)
  Raw8<BF> raw[U][R];
  uint32_t m8[U][R];
  auto fetch = [&](int64_t k0, int c0) __attribute__((always_inline)) {
    const char* const in = (const char*)(BWD ? p.grad : p.logits) + ((b * p.M + k0) * p.V + t0) * ES;
    const uint8_t* const mask =
        p.r.mask ? (const uint8_t*)(p.r.mask + b * p.r.mask_stride_b + k0 * p.r.mask_stride_m) + t0 / 8 : nullptr;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * 8 * kRuleThreads;
#pragma unroll
      for (int q = 0; q < R; ++q) {
        m8[u][q] = 0xFFu;
        if (c < tn && k0 + q < ke) {
          raw[u][q] = load8<BF, true>(in + (q * p.V + c) * ES, tn - c);
          if (mask) m8[u][q] = mask[4 * q * p.r.mask_stride_m + c / 8];
        }
      }
    }
  };
  fetch(kb, 8 * tid);  // in flight while the history is walked
  if (track) {
    const int words = keep_counts ? T / 16 + T : T / 16;
    for (int i = tid; i < words; i += kRuleThreads) rule_lds[i] = 0u;
    __syncthreads();
    count_history(p.r, b, t0, tn, seen, counts);
    // the block's tokens before those that the first group takes below
    for (int64_t i = ids ? 1 + tid : kb; i <= kb - R; i += kRuleThreads) {
      const int64_t id = ids[i];
      const uint64_t c = (uint64_t)id - (uint64_t)t0;
      if (id >= 0 && c < (uint64_t)tn) {
        atomicOr(&seen[c >> 5], 1u << (c & 31));
        if (counts) atomicAdd(&counts[c], 1u);
      }
    }
    __syncthreads();
    for (int i = tid; i < T / 32; i += kRuleThreads) any[i] = seen[i];
    __syncthreads();
  }
  for (int64_t k0 = kb; k0 < ke; k0 += R) {
    if (ids) {
      if (k0 > kb) __syncthreads();
      for (int j = tid; j < 2 * R - 1; j += kRuleThreads) {  // tokens k0 - R + 1 .. k0 + R - 1
        const int64_t at = k0 - R + 1 + j;
        const int64_t id = at >= 1 && at < p.M ? ids[at] : -1;
        const uint64_t c = (uint64_t)id - (uint64_t)t0;
        const bool mine = id >= 0 && c < (uint64_t)tn;
        if (at > k0) blk[at - k0] = mine ? (uint32_t)c : 0xFFFFFFFFu;
        if (!mine) continue;
        atomicOr(&any[c >> 5], 1u << (c & 31));
        if (at <= k0) {
          atomicOr(&seen[c >> 5], 1u << (c & 31));
          if (counts) atomicAdd(&counts[c], 1u);
        }
      }
      __syncthreads();
    }
    const int rows = (int)(ke - k0 < R ? ke - k0 : R);
    const int64_t first = (b * p.M + k0) * p.V + t0;
    const char* const lg = (const char*)p.logits + first * ES;
    char* const out = (char*)p.out + first * ES;
    for (int c0 = 8 * tid; c0 < tn; c0 += U * 8 * kRuleThreads) {
      if (k0 > kb || c0 > 8 * tid) fetch(k0, c0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 8 * kRuleThreads;
        if (c >= tn) break;
        float bias[8];
        if constexpr (!BWD)
          if (p.r.bias) bias8<8>(p.r, b * p.r.bias_stride + t0 + c, tn - c, bias);
        // what the penalties need where a bit is set, fetched before the rows
        const uint32_t a8 = track ? ((const uint8_t*)any)[c / 8] : 0u;
        uint32_t s8 = 0;
        uint32_t n8[8];
        Raw8<BF> slope[R];
        if (a8) {
          s8 = ((const uint8_t*)seen)[c / 8];
          if constexpr (BWD) {
#pragma unroll
            for (int q = 0; q < R; ++q)
              if (q < rows) slope[q] = load8<BF, false>(lg + (q * p.V + c) * ES, tn - c);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) n8[i] = counts ? counts[c + i] : 0u;
          }
        }
        uint32_t packed = 0;  // 4 bits a column: times it stands among the group's tokens so far
#pragma unroll
        for (int q = 0; q < R; ++q) {
          if (q >= rows) break;
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = raw[u][q][i];
          if (a8) {
            if (q > 0 && ids) {
              const uint32_t d = blk[q] - (uint32_t)c;
              if (d < 8u) {
                packed += 1u << (4 * d);
                s8 |= 1u << d;
              }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (s8 >> i & 1u) {
                if constexpr (BWD) x[i] = slope[q][i] > 0.0f ? x[i] / pen.repetition : x[i] * pen.repetition;
                else x[i] = pen.apply(x[i], n8[i] + (packed >> (4 * i) & 15u));
              }
          }
          if constexpr (!BWD) {
            if (p.r.bias) {
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] += bias[i];
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = (m8[u][q] >> i & 1u) ? x[i] : BWD ? 0.0f : -__builtin_inff();
          store8<BF>(out + (q * p.V + c) * ES, tn - c, x);
        }
      }
    }
  }
}

namespace {
// The call's requests from b0 on.
RulesParams requests_from(RulesParams p, int64_t b0, int64_t element) {
  const int64_t at = b0 * p.M * p.V * element;
  auto later = [](auto*& t, int64_t n) { t = t ? t + n : nullptr; };
  p.logits = (const char*)p.logits + at;
  p.grad = p.grad ? (const char*)p.grad + at : nullptr;
  p.out = (char*)p.out + at;
  p.B -= b0;
  later(p.token_ids, b0 * p.M);
  later(p.r.history, b0 * p.r.history_stride);
  later(p.r.lengths, b0);
  later(p.r.prompt_lengths, b0);
  later(p.r.repetition, b0);
  later(p.r.frequency, b0);
  later(p.r.presence, b0);
  later(p.r.mask, b0 * p.r.mask_stride_b);
  if (p.r.bias) p.r.bias = (const char*)p.r.bias + b0 * p.r.bias_stride * (p.r.bias_bf16 ? 2 : 4);
  return p;
}

template <bool BF, bool BWD>
hipError_t rules_go(const RulesParams& p, int num_cus, hipStream_t s) {
  const bool track = rules_penalise(p.r) && (p.r.history != nullptr || (p.token_ids != nullptr && p.M > 1));
  const bool keep_counts = track && !BWD && (p.r.frequency != nullptr || p.r.presence != nullptr);
  // Tiles of 2048 columns hide latency best; larger ones read the ids less
  // often, and pay when the ids outweigh the tile's logits.  T = 2048, 4096,
  // 8192, in us, bf16, V = 129280: 256 rows of one position 60, 43, 46 at
  // 2048 ids and 312, 176, 142 at 32768; 256 x 5 rows 133, 140, 149 at 256
  // ids and 438, 317, 276 at 32768.  And at least four workgroups a CU.
  int T = 2048;
  while (T < 8192 && (double)T * p.M * (BF ? 2 : 4) < 0.4 * (8.0 * (track ? p.r.history_len : 0) + 36864)) T *= 2;
  while (T > 2048 && p.B * ((p.V + T - 1) / T) < 4 * (int64_t)num_cus) T /= 2;
  const int64_t tiles = (p.V + T - 1) / T;
  const int R = p.M == 1 ? 1 : (BWD && !BF) || p.M <= 4 ? 4 : 8;
  // Few requests of many positions: spans of positions in workgroups of their
  // own, each of which counts the tokens before it, up to four workgroups a CU
  // (1 x 512 rows of 129280 in bf16, 1000 ids: 676 us as one span, 71 us so;
  // the gradient 542 and 68; 4 x 256 rows of 32000 351 and 38).
  int64_t spans = 4 * (int64_t)num_cus / (p.B * tiles);
  spans = spans < 1 ? 1 : spans;
  int64_t span = ((p.M + spans - 1) / spans + R - 1) / R * R;
  spans = (p.M + span - 1) / span;
  const size_t lds = track ? (size_t)(T / 16 + (keep_counts ? T : 0)) * 4 : 0;
  const int64_t per = kLaunchGroups / (tiles * spans);  // requests of a launch
  // Positions at a time (and vectors of columns): 1 (four), 4, 8, in us at V =
  // 129280 and 1024 ids: 256 x 1 bf16 43, 56, 56; 64 x 3 bf16 33, 30, 30; 128
  // x 8 bf16 138, 118, 110.  The gradient holds the logits of a hit beside
  // its values, which in fp32 leaves eight positions too few waves: 64 x 5 84,
  // 80, 89 and 128 x 8 244, 236, 253; in bf16 52, 47, 46 and 139, 110, 115.
  for (int64_t b0 = 0; b0 < p.B; b0 += per) {
    const RulesParams q = requests_from(p, b0, BF ? 2 : 4);
    const dim3 grid((unsigned)((q.B < per ? q.B : per) * tiles * spans)), block(kRuleThreads);
    if (R == 1)
      hipLaunchKernelGGL((logit_rules_kernel<BF, BWD, 1, 4>), grid, block, lds, s, q, T, (int)tiles, span, track, keep_counts);
    else if (R == 4)
      hipLaunchKernelGGL((logit_rules_kernel<BF, BWD, 4, 1>), grid, block, lds, s, q, T, (int)tiles, span, track, keep_counts);
    else if constexpr (!BWD || BF)
      hipLaunchKernelGGL((logit_rules_kernel<BF, BWD, 8, 1>), grid, block, lds, s, q, T, (int)tiles, span, track, keep_counts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
}  // namespace

hipError_t launch_logit_rules(const RulesParams& p, bool logits_bf16, int num_cus, hipStream_t s) {
  const bool bwd = p.grad != nullptr;
  if (logits_bf16) return bwd ? rules_go<true, true>(p, num_cus, s) : rules_go<true, false>(p, num_cus, s);
  return bwd ? rules_go<false, true>(p, num_cus, s) : rules_go<false, false>(p, num_cus, s);
}

// ---------------------------------------------------------------- left to right
namespace {
constexpr int kTableCols = 4096;  // columns of a workgroup's tile of the table
}

// The table of a request's history: as above by tiles through LDS, written
// out once.  Counts are written where the bit is set and read only there.
// 64 requests of 1024 ids at V = 129280: 7 us.
__global__ __launch_bounds__(kRuleThreads) void rule_table_kernel(TableParams p, int tiles) {
  __shared__ uint32_t seen[kTableCols / 32];
  __shared__ __attribute__((aligned(16))) uint32_t counts[kTableCols];
  const int64_t b = p.b0 + blockIdx.x / (unsigned)tiles;
  const int64_t t0 = (int64_t)(blockIdx.x % (unsigned)tiles) * kTableCols;
  const int tn = (int)(p.V - t0 < kTableCols ? p.V - t0 : kTableCols);
  const int tid = threadIdx.x;
  if (t0 == 0 && tid < kStepGroups) p.keys[tid * p.B + b] = 0u;
  for (int i = tid; i < kTableCols / 32; i += kRuleThreads) seen[i] = 0u;
  for (int i = tid; i < kTableCols / 4; i += kRuleThreads) *(u32x4_t*)&counts[4 * i] = u32x4_t{0u, 0u, 0u, 0u};
  __syncthreads();
  count_history(p.r, b, t0, tn, seen, counts);
  __syncthreads();
  const int64_t W = (p.V + 31) / 32;
  uint32_t* const gs = p.seen + b * W + t0 / 32;
  uint32_t* const gc = p.counts + b * p.V + t0;
  for (int i = tid; i < (tn + 31) / 32; i += kRuleThreads) {
    uint32_t bits = seen[i];
    gs[i] = bits;
    for (; bits; bits &= bits - 1u) {
      const int c = 32 * i + __builtin_ctz(bits);
      gc[c] = counts[c];
    }
  }
}

hipError_t launch_rule_table(const TableParams& p, hipStream_t s) {
  const int64_t tiles = (p.V + kTableCols - 1) / kTableCols;
  const int64_t per = kLaunchGroups / tiles;
  TableParams q = p;
  for (q.b0 = 0; q.b0 < p.B; q.b0 += per) {
    const int64_t n = p.B - q.b0 < per ? p.B - q.b0 : per;
    hipLaunchKernelGGL(rule_table_kernel, dim3((unsigned)(n * tiles)), dim3(kRuleThreads), 0, s, q, (int)tiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

namespace {
constexpr int kFewRows = 4;                          // rows of a workgroup of the small form
constexpr int kStepWaveCols = 64;                    // columns of a wave
constexpr int kStepCols = 4 * kStepWaveCols;         // and of a workgroup
constexpr int kStepRowBytes = 512;                   // gathered bytes of a W1 row in a chunk of the rank
constexpr int kStepPitch = kStepRowBytes + 16;       // its pitch in LDS

// The token of a row's best key of a slot.  Columns at -inf give no key, so
// none (-1) means that nothing was left; a finite value whose score at a low
// temperature is -inf gives one like any other.
__device__ __forceinline__ int64_t token_of(const uint64_t (&key)[kStepGroups]) {
  uint64_t best = 0;
#pragma unroll
  for (int g = 0; g < kStepGroups; ++g) best = max_u64(best, key[g]);
  return best != 0 ? key_index(best) : -1;
}
__device__ __forceinline__ int64_t drawn_token(const uint64_t* slot, int64_t b, int64_t B) {
  uint64_t key[kStepGroups];
#pragma unroll
  for (int g = 0; g < kStepGroups; ++g) key[g] = slot[g * B + b];
  return token_of(key);
}

// 16 bytes of a weight row from element k on (EB bytes an element), zeros past its end.
template <int EB>
__device__ __forceinline__ u32x4_t weights16(const char* row, int64_t k, int64_t rank) {
  constexpr int E = 16 / EB;
  u32x4_t w = {0u, 0u, 0u, 0u};
  if (k + E <= rank) {
    w = *(const u32x4_any_t*)(row + k * EB);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (k + e < rank) {
        if constexpr (EB == 2) w[e >> 1] |= (uint32_t)((const uint16_t*)row)[k + e] << (16 * (e & 1));
        else w[e] = ((const uint32_t*)row)[k + e];
      }
  }
  return w;
}
}  // namespace

// A workgroup: 256 columns, all rows of the step in passes of 16 RT.  The
// bias of a row tile is a product on the matrix cores with the vocabulary on
// M and the rows on N (16 x 16 blocks, bf16 or fp32 as the weights are); the
// columns of a wave's four blocks are dealt so that a lane ends up with whole
// 16-byte vectors of logits of one row, NV of them, VC columns each: 16
// consecutive columns in bf16, four quarters of the row's 64 in fp32, where a
// lane's own 64 bytes at once would spread each load over all its lines (64
// rows at V = 129280: 323 us a draft of five so, 210 us as here).  To them it adds the base
// logits (loaded before the product), applies the rules and finds the best
// score, all in registers.  W2 goes from
// memory to the operands directly (each element is used by one wave of the
// workgroup), the gathered W1 rows through LDS.
template <bool WBF, bool BF, int RT>
__global__ __launch_bounds__(256, RT == 1 ? 3 : 2) void rule_step_kernel(RuleStepParams p, int tiles, unsigned chunks) {
  constexpr int WB = WBF ? 2 : 4, KE = 16 / WB;          // bytes of a weight, weights of a 16-byte piece
  constexpr int KI = 4 * KE;                             // rank elements of a step (32 or 16)
  constexpr int KC = kStepRowBytes / WB;                 // and of a chunk
  constexpr int LB = BF ? 2 : 4, VC = 16 / LB, NV = 16 / VC;
  __shared__ __attribute__((aligned(16))) unsigned char lds_e[16 * RT * kStepPitch];
  __shared__ int64_t lds_src[16 * RT];
  __shared__ uint64_t lds_key[4][16 * RT];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int n16 = lane & 15, g4 = lane >> 4;
  // the row chunks of a column tile lie eight workgroups apart: on one XCD,
  // whose L2 then holds the tile's W2 for all of them
  const int tile = (int)(blockIdx.x / (8u * chunks)) * 8 + (int)(blockIdx.x % 8u);
  const int64_t b0 = p.b0 + (int64_t)(blockIdx.x / 8u % chunks) * 16 * RT;
  if (tile >= tiles) return;
  const int64_t V = p.V, rank = p.rank;
  const int wc0 = tile * kStepCols + kStepWaveCols * wave;  // the wave's first column (V is at most 2^30)
  // first column of the lane's vector q, and how many of its columns exist
  auto column = [&](int q) __attribute__((always_inline)) -> int {
    return BF ? wc0 + 16 * g4 + VC * q : wc0 + 4 * VC * q + VC * g4;
  };
  int have[NV];
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    const int n = (int)V - column(q);
    have[q] = n <= 0 ? 0 : n < VC ? n : VC;
  }
  // the lane's W2 rows as operands (rows past V read the last one: their sums are not used)
  const char* wrow[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int v = wc0 + (BF ? 16 * (n16 >> 2) + 4 * t + (n16 & 3) : 16 * t + n16);
    wrow[t] = (const char*)p.w2 + (v < V ? (int64_t)v : V - 1) * rank * WB;
  }
  if (tid < 16 * RT) {
    int64_t x = -1;
    if (b0 + tid < p.B) {
      if (p.k == 0) {
        x = p.first[b0 + tid];
        if (x < 0 || x >= V) {
          if (tile == 0) atomicAdd(p.bad_rows, 1u);
          x = -1;
        }
      } else {
        x = drawn_token(p.keys + ((p.k - 1) % kStepSlots) * kStepGroups * p.B, b0 + tid, p.B);
        if (tile == 0) p.tokens[(b0 + tid) * p.M + p.k - 1] = x;
      }
      if (tile == 0) {
#pragma unroll
        for (int g = 0; g < kStepGroups; ++g) p.keys[(((p.k + 1) % kStepSlots) * kStepGroups + g) * p.B + b0 + tid] = 0u;
      }
    }
    lds_src[tid] = x;
  }
  // base logits and the bits of the rules (the wave's 64 columns), on their
  // way during the product
  u32x4_t base[RT][NV];
  uint64_t mask[RT], seen[RT];
  const int W = (int)((V + 31) / 32);
  // bits of the lane's columns from a row of words: its own 16 (bf16), or the
  // wave's 64 (fp32, where they do not stand together)
  auto row_bits = [&](const uint32_t* row) __attribute__((always_inline)) -> uint64_t {
    if constexpr (BF) {
      return have[0] > 0 ? ((const uint16_t*)row)[column(0) >> 4] : 0u;
    } else {
      const int w0 = wc0 >> 5;
      return (uint64_t)(w0 < W ? row[w0] : 0u) | (uint64_t)(w0 + 1 < W ? row[w0 + 1] : 0u) << 32;
    }
  };
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t b = b0 + 16 * i + n16;
    mask[i] = ~(uint64_t)0;
    seen[i] = 0;
#pragma unroll
    for (int q = 0; q < NV; ++q) base[i][q] = u32x4_t{0u, 0u, 0u, 0u};
    if (b < p.B) {
      const char* const row = (const char*)p.base + (b * p.M + p.k) * V * LB;
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        const char* const at = row + (int64_t)column(q) * LB;
        const int n = have[q];
        if (n == VC) {
          base[i][q] = __builtin_nontemporal_load((const u32x4_any_t*)at);
        } else {
#pragma unroll
          for (int e = 0; e < VC; ++e)
            if (e < n) {
              if constexpr (BF) base[i][q][e >> 1] |= (uint32_t)((const uint16_t*)at)[e] << (16 * (e & 1));
              else base[i][q][e] = ((const uint32_t*)at)[e];
            }
        }
      }
      if (p.r.mask) mask[i] = row_bits(p.r.mask + b * p.r.mask_stride_b + p.k * p.r.mask_stride_m);
      if (p.seen) seen[i] = row_bits(p.seen + b * W);
    }
  }
  // bits of the lane's 16 columns, as they stand in its vectors
  auto own_bits = [&](uint64_t m) __attribute__((always_inline)) -> uint32_t {
    if constexpr (BF) return (uint32_t)m & 0xFFFFu;
    uint32_t o = 0;
#pragma unroll
    for (int q = 0; q < NV; ++q) o |= (uint32_t)(m >> (4 * VC * q + VC * g4) & ((1u << VC) - 1)) << (VC * q);
    return o;
  };
  f32x4_t acc[RT][4];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[i][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](int kk, const u32x4_t (&w)[4]) __attribute__((always_inline)) {  // step kk of the chunk in LDS
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const u32x4_t e = *(const u32x4_t*)&lds_e[(16 * i + n16) * kStepPitch + (4 * kk + g4) * 16];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if constexpr (WBF) {
          acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w[t]),
                                                              __builtin_bit_cast(bf16x8_t, e), acc[i][t], 0, 0, 0);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[t][j]), __uint_as_float(e[j]), acc[i][t],
                                                             0, 0, 0);
        }
      }
    }
  };
  // W2 runs two steps of the rank ahead of the products, the first of them
  // ahead of the gather
  const int whole = (int)(rank / KI);
  constexpr int SC = KC / KI;  // steps of a chunk
  u32x4_t ahead[2][4];
  auto fetch = [&](int s, u32x4_t (&w)[4]) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (s < whole) w[t] = *(const u32x4_any_t*)(wrow[t] + ((int64_t)s * KI + g4 * KE) * WB);
  };
  auto gather = [&](int64_t k0) __attribute__((always_inline)) {
    __syncthreads();  // the sources are set, and the last chunk is read
    for (int i = tid; i < 16 * RT * (kStepRowBytes / 16); i += 256) {
      const int row = i / (kStepRowBytes / 16), q = i % (kStepRowBytes / 16);
      const int64_t x = lds_src[row];
      *(u32x4_t*)&lds_e[row * kStepPitch + 16 * q] =
          x >= 0 ? weights16<WB>((const char*)p.w1 + x * rank * WB, k0 + q * KE, rank) : u32x4_t{0u, 0u, 0u, 0u};
    }
    __syncthreads();
  };
  fetch(0, ahead[0]);
  fetch(1, ahead[1]);
  for (int s = 0; s < whole; s += 2) {
    if (s % SC == 0) gather((int64_t)s * KI);
    u32x4_t w[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < 4; ++t) w[h][t] = ahead[h][t];
    fetch(s + 2, ahead[0]);
    fetch(s + 3, ahead[1]);
    multiply(s % SC, w[0]);
    if (s + 1 < whole) multiply(s % SC + 1, w[1]);
  }
  if ((int64_t)whole * KI < rank) {  // the rest of a rank that is no whole number of steps
    if (whole % SC == 0) gather((int64_t)whole * KI);
    u32x4_t w[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) w[t] = weights16<WB>(wrow[t], (int64_t)whole * KI + g4 * KE, rank);
    multiply(whole % SC, w);
  }
  // counts of the columns that stand in the table, a row tile ahead of their use
  uint32_t count[2][16];
  auto fetch_counts = [&](int i) __attribute__((always_inline)) {
    if (i < RT && own_bits(seen[i < RT ? i : 0])) {
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        const u32x4_t w = *(const u32x4_any_t*)(p.counts + (b0 + 16 * i + n16) * V + column(4 * e4 / VC) + 4 * e4 % VC);
#pragma unroll
        for (int e = 0; e < 4; ++e) count[i & 1][4 * e4 + e] = w[e];
      }
    }
  };
  fetch_counts(0);
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t b = b0 + 16 * i + n16;
    fetch_counts(i + 1);
    uint32_t s16 = own_bits(seen[i]);
    const uint32_t m16 = own_bits(mask[i]);
    if (p.seen && p.k > 0) {
      // the token of the last position joins the table in the one lane, of all
      // the step's workgroups, that has its column
      const int64_t t = lds_src[16 * i + n16];
      const int rel = (int)(t - wc0);
      if (t >= wc0 && rel < kStepWaveCols && (BF ? rel >> 4 : rel >> 2 & 3) == g4) {
        const int mine = BF ? rel & 15 : 4 * (rel >> 4) + (rel & 3);
        uint32_t n = 1u;
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (e == mine) count[i & 1][e] = n = (s16 >> e & 1u) ? count[i & 1][e] + 1u : 1u;
        s16 |= 1u << mine;
        p.counts[b * V + t] = n;
        if constexpr (BF) ((uint16_t*)(p.seen + b * W))[t >> 4] = (uint16_t)s16;
        else p.seen[b * W + (t >> 5)] = (uint32_t)(seen[i] >> (rel & 32)) | 1u << (t & 31);
      }
    }
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float bias = acc[i][e >> 2][e & 3];
      if constexpr (WBF || BF) bias = bf16_rne(bias);
      if constexpr (BF) {
        const uint32_t w = base[i][e >> 3][e >> 1 & 3];
        x[e] = bf16_rne(((e & 1) ? bf16_hi(w) : bf16_lo(w)) + bias);
      } else {
        x[e] = __uint_as_float(base[i][e >> 2][e & 3]) + bias;
      }
    }
    if (s16) {
      const Penalty pen = penalty_of(p.r, b);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (s16 >> e & 1u) x[e] = pen.apply(x[e], count[i & 1][e]);
    }
    uint64_t best = 0;
    if (b < p.B) {
      if (p.r.bias) {
#pragma unroll
        for (int q = 0; q < NV; ++q) {
          float bias[8];
          bias8<VC>(p.r, b * p.r.bias_stride + column(q), have[q], bias);
#pragma unroll
          for (int e = 0; e < VC; ++e) x[VC * q + e] += bias[e];
        }
      }
      char* const row = (char*)p.out + (b * p.M + p.k) * V * LB;
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        const int n = have[q];
        u32x4_t w;
#pragma unroll
        for (int e = 0; e < VC; ++e) {
          float& y = x[VC * q + e];
          y = (m16 >> (VC * q + e) & 1u) ? y : -__builtin_inff();
          if constexpr (BF) y = bf16_rne(y);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (BF) w[e] = join_bf16(x[VC * q + 2 * e], x[VC * q + 2 * e + 1]);
          else w[e] = __float_as_uint(x[VC * q + e]);
        }
        char* const at = row + (int64_t)column(q) * LB;
        if (n == VC) {
          __builtin_nontemporal_store(w, (u32x4_any_t*)at);
        } else {
#pragma unroll
          for (int e = 0; e < VC; ++e)
            if (e < n) {
              if constexpr (BF) ((uint16_t*)at)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
              else ((uint32_t*)at)[e] = w[e];
            }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // groups of four columns: the words of one noise block
        const int v = column(4 * j / VC) + 4 * j % VC;
        float g[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (!p.greedy) {
          const Philox4 q = philox4x32_10((uint32_t)(v >> 2), p.k_abs, (uint32_t)p.batch_offset + (uint32_t)b, 0u,
                                          p.seed_lo, p.seed_hi);
          g[0] = gumbel2_from_word(q.x0);
          g[1] = gumbel2_from_word(q.x1);
          g[2] = gumbel2_from_word(q.x2);
          g[3] = gumbel2_from_word(q.x3);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float sc = p.greedy ? x[4 * j + e] : __builtin_fmaf(x[4 * j + e], p.kappa, g[e]);
          if (4 * j % VC + e < have[4 * j / VC] && x[4 * j + e] != -__builtin_inff())
            best = max_u64(best, argmax_key(sc, (uint32_t)(v + e)));
        }
      }
    }
    best = max_row_lanes(best);
    if (lane < 16) lds_key[wave][16 * i + lane] = best;
  }
  __syncthreads();
  const bool row_ok = tid < 16 * RT && b0 + tid < p.B;
  uint64_t best = 0;
  if (row_ok) best = max_u64(max_u64(lds_key[0][tid], lds_key[1][tid]), max_u64(lds_key[2][tid], lds_key[3][tid]));
  if (row_ok)
    __hip_atomic_fetch_max(p.keys + ((p.k % kStepSlots) * kStepGroups + tile % kStepGroups) * p.B + b0 + tid, best,
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The same step by four rows a workgroup.  With the rows on the matrix
// instruction's 16 columns most lanes would hold rows that do not exist and
// the others 16 columns each, a long stretch of code for a lone wave of a SIMD;
// here a lane ends up with four consecutive columns of one row: a vector of
// logits and a block of noise.  A row's sums are those of the kernel above to
// the bit, so that a batch may be cut anywhere.  In bf16 that takes the same
// instruction, whose order of the sum within its 32 elements no smaller one
// has: the four rows stand four times on its columns, and a lane takes the
// block of its own columns.  The fp32 instruction above sums its four elements
// one after the other, as 4 x 4 blocks do that go through them in that order.
// Both operands go to registers, two lines of 128 bytes of a row ahead of the
// products, and nothing waits at a barrier before the keys.
// W2 is loaded a line by eight lanes and turned through LDS: lanes loading
// their own rows touch a line each (rank 256 in fp32, V = 129280, drafts of
// five: 1 row 162 us so, 139 us as here, 146 us by the kernel above; 4 rows
// 189, 143 and 136 us; in bf16 97 us a draft by 4 x 4 x 4 products, 83 us as
// here).  Bound by latency where W2 is short: V = 50257 at rank 64 in fp32
// 8.3 us a step, 12.2 us by the kernel above.  More rows take more
// workgroups, each reading its columns of W2, from the XCD's L2; two sets of
// blocks in one wave took 52 -> 71 us a draft instead (8 rows, V = 32000).
template <bool WBF, bool BF, bool RAGGED>
__global__ __launch_bounds__(256, 2) void rule_few_kernel(RuleStepParams p, int tiles, unsigned chunks) {
  constexpr int WB = WBF ? 2 : 4, KE = 16 / WB, KI = 4 * KE;  // as above
  constexpr int LB = BF ? 2 : 4, NP = 8;                      // bytes of a logit, pieces of a line (two steps of KI)
  constexpr int NE = WBF ? 2 : NP;                            // pieces of a row's line that a lane supplies
  typedef uint32_t base_t __attribute__((ext_vector_type(LB), aligned(2)));
  __shared__ uint64_t lds_key[4][kFewRows];
  __shared__ __attribute__((aligned(16))) unsigned char lds_w[4][kStepWaveCols * 128];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int tile = (int)(blockIdx.x / (8u * chunks)) * 8 + (int)(blockIdx.x % 8u);
  const int64_t b0 = (int64_t)(blockIdx.x / 8u % chunks) * kFewRows;
  if (tile >= tiles) return;
  const int64_t V = p.V, rank = p.rank, W = (V + 31) / 32, b = b0 + (lane & 3);
  const int wc0 = tile * kStepCols + kStepWaveCols * wave, c0 = wc0 + (lane & ~3);  // V is at most 2^30
  const int left = (int)V - c0, have = left < 0 ? 0 : left < 4 ? left : 4;
  const int steps = (int)((rank + KI - 1) / KI), lines = (steps + 1) / 2, pieces = (int)((rank + KE - 1) / KE);
  // The last piece of a rank that is no whole number of them is loaded as the
  // row's last 16 bytes and moved down when it is used, with zeros behind it.
  auto piece_at = [&](int piece) __attribute__((always_inline)) { return RAGGED ? min(16 * piece, (int)rank * WB - 16) : 16 * piece; };
  auto settle = [&](const u32x4_t& d, int piece) __attribute__((always_inline)) -> u32x4_t {
    const int bits = 8 * (16 * piece - piece_at(piece)), n = bits & 63;
    const uint64_t lo = bits < 64 ? (uint64_t)d[1] << 32 | d[0] : (uint64_t)d[3] << 32 | d[2];
    const uint64_t hi = bits < 64 ? (uint64_t)d[3] << 32 | d[2] : 0u;
    const uint64_t a = n ? lo >> n | hi << (64 - n) : lo, b = hi >> n;
    return u32x4_t{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)};
  };
  uint64_t key[kStepGroups];
  int64_t x = -1;  // the row's predecessor
  if (b < p.B) {
    if (p.k == 0) {
      x = p.first[b];
    } else {
#pragma unroll
      for (int i = 0; i < kStepGroups; ++i) key[i] = p.keys[(((p.k - 1) % kStepSlots) * kStepGroups + i) * p.B + b];
    }
  }
  // W2, its first lines ahead of everything that waits: load i of a line takes
  // rows 8 i .. 8 i + 7 of the wave's (past V: the last row)
  auto row_of = [&](int i) __attribute__((always_inline)) -> const char* {
    const int64_t v = wc0 + i < V ? wc0 + i : V - 1;
    return (const char*)p.w2 + v * rank * WB;
  };
  const int pc = lane & 7, r8 = lane >> 3, n16 = lane & 15, g4 = lane >> 4;
  u32x4_t w[2][NP], e[2][NE];
  auto fetch_w = [&](int l, u32x4_t (&d)[NP]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      d[i] = u32x4_t{0u, 0u, 0u, 0u};
      if (NP * l + pc < pieces) d[i] = *(const u32x4_any_t*)(row_of(8 * i + r8) + piece_at(NP * l + pc));
    }
  };
  // a line's operands out of its loads, through the wave's own LDS (a wave's
  // LDS accesses keep their order): bf16, piece 4 h + g4 of the rows that stand
  // at n16 in blocks t = 0 .. 3, at 4 h + t; fp32, the lane's own row.  Pieces
  // are swizzled so that rows read together fall on different banks.
  unsigned char* const mine = lds_w[wave];
  auto block_row = [&](int t) __attribute__((always_inline)) { return 16 * (n16 >> 2) + 4 * t + (n16 & 3); };
  auto turn = [&](const u32x4_t (&d)[NP], u32x4_t (&a)[NP]) __attribute__((always_inline)) {
    auto place = [&](int row, int piece) __attribute__((always_inline)) {
      return (u32x4_t*)(mine + row * 128 + 16 * (piece ^ (WBF ? (row & 3) | (row >> 4 & 1) << 2 : row & 7)));
    };
#pragma unroll
    for (int i = 0; i < NP; ++i) *place(8 * i + r8, pc) = d[i];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < NP; ++q) a[q] = WBF ? *place(block_row(q & 3), 4 * (q >> 2) + g4) : *place(lane, q);
    __builtin_amdgcn_wave_barrier();
  };
  fetch_w(0, w[0]);
  fetch_w(1, w[1]);
  // base logits and what the rules need of the lane's columns
  uint32_t raw[4] = {0u, 0u, 0u, 0u}, seen = 0u, mask = ~0u, word = 0u;
  float bias[8];
  Penalty pen{};
  if (b < p.B && have > 0) {
    const char* const at = (const char*)p.base + ((b * p.M + p.k) * V + c0) * LB;
    if (have == 4) {
      const base_t d = __builtin_nontemporal_load((const base_t*)at);
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[i] = BF ? (i & 1 ? d[i >> 1] >> 16 : d[i >> 1] & 0xFFFFu) : d[i & (LB - 1)];
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < have) raw[i] = BF ? ((const uint16_t*)at)[i] : ((const uint32_t*)at)[i];
    }
    if (p.seen) {
      word = p.seen[b * W + (c0 >> 5)];
      pen = penalty_of(p.r, b);
    }
    if (p.r.mask) mask = p.r.mask[b * p.r.mask_stride_b + p.k * p.r.mask_stride_m + (c0 >> 5)];
    if (p.r.bias) bias8<4>(p.r, b * p.r.bias_stride + c0, have, bias);
  }
  // the predecessor, and the next step's slot
  if (b < p.B) {
    const bool writer = tile == 0 && tid < kFewRows;
    if (p.k == 0) {
      if (x < 0 || x >= V) {
        if (writer) atomicAdd(p.bad_rows, 1u);
        x = -1;
      }
    } else {
      x = token_of(key);
      if (writer) p.tokens[b * p.M + p.k - 1] = x;
    }
    if (writer) {
#pragma unroll
      for (int i = 0; i < kStepGroups; ++i) p.keys[(((p.k + 1) % kStepSlots) * kStepGroups + i) * p.B + b] = 0u;
    }
  }
  const char* const erow = (const char*)p.w1 + (x < 0 ? 0 : x) * rank * WB;
  auto fetch_e = [&](int l, u32x4_t (&d)[NE]) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < NE; ++q) {
      const int piece = NP * l + (WBF ? 4 * q + g4 : q);
      d[q] = u32x4_t{0u, 0u, 0u, 0u};
      if (piece < pieces && x >= 0) d[q] = *(const u32x4_any_t*)(erow + piece_at(piece));
    }
  };
  fetch_e(0, e[0]);
  fetch_e(1, e[1]);
  // counts of the lane's columns that stand in the table, and the last
  // position's token, which joins it in the one lane of all the step's
  // workgroups that has its column
  uint32_t count[4];
  seen = word >> (c0 & 31) & 15u;
  if (seen) {
    const u32x4_t n = *(const u32x4_any_t*)(p.counts + b * V + c0);
#pragma unroll
    for (int i = 0; i < 4; ++i) count[i] = n[i];
  }
  if (p.seen && p.k > 0 && x >= c0 && x < c0 + 4) {
    const int at = (int)x - c0;
    uint32_t n = 1u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i == at) count[i] = n = (seen >> i & 1u) ? count[i] + 1u : 1u;
    seen |= 1u << at;
    p.counts[b * V + x] = n;
    p.seen[b * W + (c0 >> 5)] = word | 1u << (x & 31);
  }
  constexpr int NA = WBF ? 4 : 1;  // blocks of sums
  f32x4_t acc[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  // a step of KI: in fp32 element j of each of its pieces in turn, as above
  auto multiply = [&](const u32x4_t* wp, const u32x4_t* ep) __attribute__((always_inline)) {
    if constexpr (WBF) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, wp[t]),
                                                         __builtin_bit_cast(bf16x8_t, ep[0]), acc[t], 0, 0, 0);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          acc[0] = __builtin_amdgcn_mfma_f32_4x4x1f32(__uint_as_float(wp[g][j]), __uint_as_float(ep[g][j]), acc[0], 0, 0, 0);
    }
  };
  for (int l = 0; l < lines; l += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (l + h < lines) {
        u32x4_t a[NP];
        if (RAGGED && l + h == lines - 1) {
#pragma unroll
          for (int i = 0; i < NP; ++i)
            if (NP * (l + h) + pc == pieces - 1) w[h][i] = settle(w[h][i], pieces - 1);
#pragma unroll
          for (int q = 0; q < NE; ++q)
            if (NP * (l + h) + (WBF ? 4 * q + g4 : q) == pieces - 1) e[h][q] = settle(e[h][q], pieces - 1);
        }
        turn(w[h], a);
        multiply(a, e[h]);
        if (2 * (l + h) + 1 < steps) multiply(a + 4, e[h] + NE / 2);
        if (l + h + 2 < lines) {
          fetch_w(l + h + 2, w[h]);
          fetch_e(l + h + 2, e[h]);
        }
      }
  }
  uint64_t best = 0;
  if (b < p.B && have > 0) {
    f32x4_t sum = acc[0];  // of the block whose columns are the lane's
#pragma unroll
    for (int t = 1; t < NA; ++t) sum = n16 >> 2 == t ? acc[t] : sum;
    float y[4], noise[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (!p.greedy) {
      const Philox4 q = philox4x32_10((uint32_t)(c0 >> 2), p.k_abs, (uint32_t)p.batch_offset + (uint32_t)b, 0u, p.seed_lo,
                                      p.seed_hi);
      noise[0] = gumbel2_from_word(q.x0);
      noise[1] = gumbel2_from_word(q.x1);
      noise[2] = gumbel2_from_word(q.x2);
      noise[3] = gumbel2_from_word(q.x3);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float product = WBF || BF ? bf16_rne(sum[i]) : sum[i];
      y[i] = BF ? bf16_rne(bf16_lo(raw[i]) + product) : __uint_as_float(raw[i]) + product;
      if (seen >> i & 1u) y[i] = pen.apply(y[i], count[i]);
      if (p.r.bias) y[i] += bias[i];
      y[i] = (mask >> ((c0 & 31) + i) & 1u) ? y[i] : -__builtin_inff();
      if (BF) y[i] = bf16_rne(y[i]);
      const float sc = p.greedy ? y[i] : __builtin_fmaf(y[i], p.kappa, noise[i]);
      if (i < have && y[i] != -__builtin_inff()) best = max_u64(best, argmax_key(sc, (uint32_t)(c0 + i)));
    }
    char* const at = (char*)p.out + ((b * p.M + p.k) * V + c0) * LB;
    if (have == 4) {
      base_t d;
      if constexpr (BF) {
        d[0] = join_bf16(y[0], y[1]);
        d[1] = join_bf16(y[2], y[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = __float_as_uint(y[i]);
      }
      __builtin_nontemporal_store(d, (base_t*)at);
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < have) {
          if constexpr (BF) ((uint16_t*)at)[i] = (uint16_t)(__float_as_uint(y[i]) >> 16);
          else ((float*)at)[i] = y[i];
        }
    }
  }
  best = max_u64(best, __shfl_xor(best, 4));
  best = max_u64(best, __shfl_xor(best, 8));
  best = max_row_lanes(best);
  if (lane < kFewRows) lds_key[wave][lane] = best;
  __syncthreads();
  if (tid < kFewRows && b0 + tid < p.B)
    __hip_atomic_fetch_max(p.keys + ((p.k % kStepSlots) * kStepGroups + tile % kStepGroups) * p.B + b0 + tid,
                           max_u64(max_u64(lds_key[0][tid], lds_key[1][tid]), max_u64(lds_key[2][tid], lds_key[3][tid])),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

namespace {
template <bool WBF, bool BF, int RT>
hipError_t rule_step_form(const RuleStepParams& p, hipStream_t s) {
  const int64_t tiles = (p.V + kStepCols - 1) / kStepCols, columns = (tiles + 7) / 8 * 8;
  const int64_t per = kLaunchGroups / columns * 16 * RT;  // rows of a launch
  RuleStepParams q = p;
  for (q.b0 = 0; q.b0 < p.B; q.b0 += per) {
    const int64_t chunks = ((p.B - q.b0 < per ? p.B - q.b0 : per) + 16 * RT - 1) / (16 * RT);
    hipLaunchKernelGGL((rule_step_kernel<WBF, BF, RT>), dim3((unsigned)(columns * chunks)), dim3(256), 0, s, q, (int)tiles,
                       (unsigned)chunks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <bool WBF, bool BF>
hipError_t rule_few_form(const RuleStepParams& p, hipStream_t s) {
  const int64_t tiles = (p.V + kStepCols - 1) / kStepCols, chunks = (p.B + kFewRows - 1) / kFewRows;
  const dim3 grid((unsigned)((tiles + 7) / 8 * 8 * chunks)), block(256);
  if (p.rank % (WBF ? 8 : 4) == 0)
    hipLaunchKernelGGL((rule_few_kernel<WBF, BF, false>), grid, block, 0, s, p, (int)tiles, (unsigned)chunks);
  else
    hipLaunchKernelGGL((rule_few_kernel<WBF, BF, true>), grid, block, 0, s, p, (int)tiles, (unsigned)chunks);
  return hipGetLastError();
}
template <bool WBF, bool BF>
hipError_t rule_step_go(const RuleStepParams& p, int num_cus, hipStream_t s) {
  // whether the device holds all workgroups of so many rows at once
  auto fits = [&](int64_t rows) { return (p.V + kStepCols - 1) / kStepCols * ((p.B + rows - 1) / rows) <= 2 * (int64_t)num_cus; };
  // Four rows a workgroup while the device holds all of them at once (two a
  // CU), or there are no more rows; otherwise the fewer readers of W2.  In us,
  // drafts of five, so and by the kernel for row tiles: 250 workgroups (8 rows,
  // V = 32000, rank 64, bf16) 39, 52; 256 (64 rows, V = 4000, rank 64, fp32)
  // 47, 178; 500 (16 rows, V = 32000) 41, 55; 1010 (8 rows, V = 129280) 74, 58.
  // Beyond a drafter's 64 rows it is not measured; rows of less than 16 bytes
  // have no whole piece to load.  The form does not change a row's sums.
  if (p.rank >= (WBF ? 8 : 4) && (p.B <= kFewRows || (p.B <= 64 && fits(kFewRows)))) return rule_few_form<WBF, BF>(p, s);
  // Row tiles a workgroup: the fewest with which the device holds all
  // workgroups at once, as each waits for the same loads however few its
  // tiles; at most four, and no more than there are.  In us, drafts of five at
  // rank 256 in bf16 with one, two and four: 32 rows, V = 32000 72, 100, 105;
  // 64 rows, V = 32000 93, 101, 157, V = 65536 157, 122, 160, V = 100000 220,
  // 204, 176; 256 rows, V = 16000 157, 130, 161; 54 rows, V = 29826 in fp32
  // 143, 145, 247.
  if (p.B <= 16 || fits(16)) return rule_step_form<WBF, BF, 1>(p, s);
  if (p.B <= 32 || fits(32)) return rule_step_form<WBF, BF, 2>(p, s);
  return rule_step_form<WBF, BF, 4>(p, s);
}
}  // namespace

hipError_t launch_rule_step(const RuleStepParams& p, bool logits_bf16, bool weights_bf16, int num_cus, hipStream_t s) {
  if (weights_bf16) return logits_bf16 ? rule_step_go<true, true>(p, num_cus, s) : rule_step_go<true, false>(p, num_cus, s);
  return logits_bf16 ? rule_step_go<false, true>(p, num_cus, s) : rule_step_go<false, false>(p, num_cus, s);
}

__global__ __launch_bounds__(kRuleThreads) void rule_choose_kernel(const uint64_t* __restrict__ slot, int64_t B, int64_t M,
                                                                   int64_t* __restrict__ tokens) {
  const int64_t b = (int64_t)blockIdx.x * kRuleThreads + threadIdx.x;
  if (b < B) tokens[b * M + M - 1] = drawn_token(slot, b, B);
}

hipError_t launch_rule_choose(const uint64_t* keys, int64_t B, int64_t M, int64_t* tokens, hipStream_t s) {
  const int64_t groups = (B + kRuleThreads - 1) / kRuleThreads;
  if (groups > kLaunchGroups) return hipErrorNotSupported;
  hipLaunchKernelGGL(rule_choose_kernel, dim3((unsigned)groups), dim3(kRuleThreads), 0, s,
                     keys + ((M - 1) % kStepSlots) * kStepGroups * B, B, M, tokens);
  return hipGetLastError();
}

}  // namespace dspark
