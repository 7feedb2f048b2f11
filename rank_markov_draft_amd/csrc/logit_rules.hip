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
// tile of all M positions past that table.  The ids are re-read once per tile
// of the vocabulary, from L2; nothing is sorted or written to memory.
#include "device_common.h"
#include "logit_rules.h"

namespace dspark {

namespace {

constexpr int kRuleThreads = 256;

// Bits c .. c + 7 of a bitmap of n words (c may lie outside: zeros there).
__device__ __forceinline__ uint32_t bits8(const uint32_t* w, int n, int c) {
  const int i = c >> 5;
  const uint32_t lo = (uint32_t)i < (uint32_t)n ? w[i] : 0u;
  const uint32_t hi = (uint32_t)(i + 1) < (uint32_t)n ? w[i + 1] : 0u;
  return (uint32_t)((((uint64_t)hi << 32) | lo) >> (c & 31)) & 0xFFu;
}

__device__ __forceinline__ float bias_at(const RuleSet& r, int64_t i) {
  return r.bias_bf16 ? bf16_lo(((const uint16_t*)r.bias)[i]) : ((const float*)r.bias)[i];
}

// A request's penalties; a rule that is off leaves x as it is.
struct Penalty {
  float repetition, frequency, presence;
  bool repeat, count;
  __device__ __forceinline__ float apply(float x, uint32_t c) const {
    if (repeat) x = x > 0.0f ? x / repetition : x * repetition;
    if (count && c > 0u) x = x - (frequency * (float)c + presence);
    return x;
  }
};
__device__ __forceinline__ Penalty penalty_of(const RuleSet& r, int64_t b) {
  return Penalty{r.repetition ? r.repetition[b] : 1.0f, r.frequency ? r.frequency[b] : 0.0f,
                 r.presence ? r.presence[b] : 0.0f, r.repetition != nullptr,
                 r.frequency != nullptr || r.presence != nullptr};
}

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

// The 8 values at columns c .. c + 7 of a row; `full`: all of them exist and
// the vector may be loaded whole, else those with c + i in [0, n).
template <bool BF>
__device__ __forceinline__ void load8(const void* row, int c, int n, bool full, float (&x)[8]) {
  if (full) {
    if constexpr (BF) {
      const u32x4_t w = __builtin_nontemporal_load((const u32x4_t*)((const uint16_t*)row + c));
      const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(q[i]);
        x[2 * i + 1] = bf16_hi(q[i]);
      }
    } else {
      const f32x4_t a = __builtin_nontemporal_load((const f32x4_t*)((const float*)row + c));
      const f32x4_t b = __builtin_nontemporal_load((const f32x4_t*)((const float*)row + c + 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = a[i];
        x[4 + i] = b[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = 0.0f;
      if ((uint32_t)(c + i) < (uint32_t)n)
        x[i] = BF ? bf16_lo(((const uint16_t*)row)[c + i]) : ((const float*)row)[c + i];
    }
  }
}
template <bool BF>
__device__ __forceinline__ void store8(void* row, int c, int n, bool full, const float (&x)[8]) {
  if (full) {
    if constexpr (BF) {
      const u32x4_t w = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                         pack_bf16x2(x[6], x[7])};
      __builtin_nontemporal_store(w, (u32x4_t*)((uint16_t*)row + c));
    } else {
      __builtin_nontemporal_store(f32x4_t{x[0], x[1], x[2], x[3]}, (f32x4_t*)((float*)row + c));
      __builtin_nontemporal_store(f32x4_t{x[4], x[5], x[6], x[7]}, (f32x4_t*)((float*)row + c + 4));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((uint32_t)(c + i) < (uint32_t)n) {
        if constexpr (BF) ((uint16_t*)row)[c + i] = (uint16_t)(pack_bf16x2(x[i], 0.0f) & 0xFFFFu);
        else ((float*)row)[c + i] = x[i];
      }
  }
}

}  // namespace

// T columns of one request a workgroup, all its positions.  Rows of an odd
// vocabulary start anywhere, so each row's vectors of 8 are laid from the
// 16-byte boundary at or before the tile's first column; a vector that
// reaches past the tile is moved by elements.  `whole` is false where the
// streamed tensors differ in alignment: then every vector is.
template <bool BF, bool BWD>
__global__ __launch_bounds__(kRuleThreads) void logit_rules_kernel(RulesParams p, int T, int tiles, bool track,
                                                                   bool keep_counts, bool whole) {
  extern __shared__ uint32_t rule_lds[];
  uint32_t* const seen = rule_lds;                                    // T / 32 words
  uint32_t* const counts = keep_counts ? rule_lds + T / 32 : nullptr;  // T words
  const int64_t b = blockIdx.x / (unsigned)tiles;
  const int64_t t0 = (int64_t)(blockIdx.x % (unsigned)tiles) * T;
  const int tn = (int)(p.V - t0 < T ? p.V - t0 : T);
  const int tid = threadIdx.x;
  constexpr int ES = BF ? 2 : 4;
  const Penalty pen = penalty_of(p.r, b);
  if (track) {
    const int words = keep_counts ? T / 32 + T : T / 32;
    for (int i = tid; i < words; i += kRuleThreads) rule_lds[i] = 0u;
    __syncthreads();
    count_history(p.r, b, t0, tn, seen, counts);
    __syncthreads();
  }
  const int W = (int)((p.V + 31) / 32);
  for (int64_t k = 0; k < p.M; ++k) {
    if (track && k > 0 && p.token_ids) {
      // the block's token before this position, if it is the tile's
      const int64_t id = p.token_ids[b * p.M + k];
      const uint64_t c = (uint64_t)id - (uint64_t)t0;
      if (id >= 0 && c < (uint64_t)tn) {  // the same in every thread
        __syncthreads();
        if (tid == 0) {
          seen[c >> 5] |= 1u << (c & 31);
          if (counts) counts[c] += 1u;
        }
        __syncthreads();
      }
    }
    const int64_t row = (b * p.M + k) * p.V + t0;
    const char* const in = (const char*)(BWD ? p.grad : p.logits) + row * ES;
    char* const out = (char*)p.out + row * ES;
    const char* const lg = (const char*)p.logits + row * ES;
    const int a = whole ? (int)(((uintptr_t)out % 16) / ES) : 0;
    const uint32_t* const mask = p.r.mask ? p.r.mask + b * p.r.mask_stride_b + k * p.r.mask_stride_m : nullptr;
    const int64_t bias0 = b * p.r.bias_stride + t0;
    constexpr int U = 2;
    for (int c0 = 8 * tid - a; c0 < tn; c0 += U * 8 * kRuleThreads) {
      float x[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 8 * kRuleThreads;
        if (c < tn) load8<BF>(in, c, tn, whole && c >= 0 && c + 8 <= tn, x[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 8 * kRuleThreads;
        if (c >= tn) break;
        const uint32_t s8 = track ? bits8(seen, T / 32, c) : 0u;
        if (s8) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (s8 >> i & 1u) {
              if constexpr (BWD) {
                const float l = BF ? bf16_lo(((const uint16_t*)lg)[c + i]) : ((const float*)lg)[c + i];
                x[u][i] = l > 0.0f ? x[u][i] / pen.repetition : x[u][i] * pen.repetition;
              } else {
                x[u][i] = pen.apply(x[u][i], counts ? counts[c + i] : 0u);
              }
            }
        }
        if constexpr (!BWD) {
          if (p.r.bias) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if ((uint32_t)(c + i) < (uint32_t)tn) x[u][i] += bias_at(p.r, bias0 + c + i);
          }
        }
        if (mask) {
          const uint32_t m8 = bits8(mask, W, (int)t0 + c);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[u][i] = (m8 >> i & 1u) ? x[u][i] : BWD ? 0.0f : -__builtin_inff();
        }
        store8<BF>(out, c, tn, whole && c >= 0 && c + 8 <= tn, x[u]);
      }
    }
  }
}

hipError_t launch_logit_rules(const RulesParams& p, bool logits_bf16, int num_cus, hipStream_t s) {
  const bool track = rules_penalise(p.r) && (p.r.history != nullptr || (p.token_ids != nullptr && p.M > 1));
  const bool bwd = p.grad != nullptr;
  const bool keep_counts = track && !bwd && (p.r.frequency != nullptr || p.r.presence != nullptr);
  int T = 8192;
  while (T > 2048 && p.B * ((p.V + T - 1) / T) < 4 * (int64_t)num_cus) T /= 2;
  const int64_t tiles = (p.V + T - 1) / T;
  if (p.B * tiles > 0x7FFFFFFF) return hipErrorNotSupported;
  const size_t lds = track ? (size_t)(T / 32 + (keep_counts ? T : 0)) * 4 : 0;
  const bool whole = ((uintptr_t)(bwd ? p.grad : p.logits) - (uintptr_t)p.out) % 16 == 0;
  const dim3 grid((unsigned)(p.B * tiles)), block(kRuleThreads);
#define DSPARK_RULES(BF, BWD) \
  hipLaunchKernelGGL((logit_rules_kernel<BF, BWD>), grid, block, lds, s, p, T, (int)tiles, track, keep_counts, whole)
  if (logits_bf16) {
    if (bwd) DSPARK_RULES(true, true);
    else DSPARK_RULES(true, false);
  } else {
    if (bwd) DSPARK_RULES(false, true);
    else DSPARK_RULES(false, false);
  }
#undef DSPARK_RULES
  return hipGetLastError();
}

// ---------------------------------------------------------------- left to right
namespace {
constexpr int kTableCols = 8192;  // columns of a workgroup's tile of the table
}

// The table of a request's history: as above by tiles through LDS, written
// out once.  Counts are written where the bit is set and read only there.
__global__ __launch_bounds__(kRuleThreads) void rule_table_kernel(TableParams p, int tiles) {
  __shared__ uint32_t seen[kTableCols / 32];
  __shared__ uint32_t counts[kTableCols];
  const int64_t b = blockIdx.x / (unsigned)tiles;
  const int64_t t0 = (int64_t)(blockIdx.x % (unsigned)tiles) * kTableCols;
  const int tn = (int)(p.V - t0 < kTableCols ? p.V - t0 : kTableCols);
  const int tid = threadIdx.x;
  for (int i = tid; i < kTableCols / 32; i += kRuleThreads) seen[i] = 0u;
  for (int i = tid; i < kTableCols; i += kRuleThreads) counts[i] = 0u;
  __syncthreads();
  count_history(p.r, b, t0, tn, seen, counts);
  __syncthreads();
  const int64_t W = (p.V + 31) / 32;
  uint32_t* const gs = p.seen + b * W + t0 / 32;
  uint32_t* const gc = p.counts + b * p.V + t0;
  for (int i = tid; i < (tn + 31) / 32; i += kRuleThreads) gs[i] = seen[i];
  for (int i = tid; i < tn; i += kRuleThreads)
    if (seen[i >> 5] >> (i & 31) & 1u) gc[i] = counts[i];
}

hipError_t launch_rule_table(const TableParams& p, int num_cus, hipStream_t s) {
  (void)num_cus;
  const int64_t tiles = (p.V + kTableCols - 1) / kTableCols;
  if (p.B * tiles > 0x7FFFFFFF) return hipErrorNotSupported;
  hipLaunchKernelGGL(rule_table_kernel, dim3((unsigned)(p.B * tiles)), dim3(kRuleThreads), 0, s, p, (int)tiles);
  return hipGetLastError();
}

namespace {
constexpr int kSelectCols = 4096;  // columns of a workgroup's slice of a row
}
int64_t select_parts(int64_t V) { return (V + kSelectCols - 1) / kSelectCols; }

// One row's slice: the rules in place, then the slice's best key (the scores
// of sample_block_tokens on the processed values).
template <bool BF>
__global__ __launch_bounds__(kRuleThreads) void rule_select_kernel(SelectParams p, int parts, bool whole) {
  __shared__ uint64_t lds_key[kRuleThreads / 64];
  const int64_t b = blockIdx.x / (unsigned)parts;
  const int part = (int)(blockIdx.x % (unsigned)parts);
  const int tid = threadIdx.x;
  const int V = (int)p.V;
  const int end = V - part * kSelectCols < kSelectCols ? V : (part + 1) * kSelectCols;
  const int W = (V + 31) / 32;
  const Penalty pen = penalty_of(p.r, b);
  char* const row = (char*)p.logits + (b * p.M + p.k) * p.V * (BF ? 2 : 4);
  const uint32_t* const seen = p.seen ? p.seen + b * W : nullptr;
  const uint32_t* const counts = p.seen ? p.counts + b * p.V : nullptr;
  const uint32_t* const mask = p.r.mask ? p.r.mask + b * p.r.mask_stride_b + p.k * p.r.mask_stride_m : nullptr;
  const int64_t bias0 = b * p.r.bias_stride;
  uint64_t best = 0;
  constexpr int U = kSelectCols / (8 * kRuleThreads);
  float x[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = part * kSelectCols + 8 * (tid + u * kRuleThreads);
    if (c < end) load8<BF>(row, c, V, whole && c + 8 <= V, x[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = part * kSelectCols + 8 * (tid + u * kRuleThreads);
    if (c >= end) break;
    const uint32_t s8 = seen ? bits8(seen, W, c) : 0u;
    if (s8) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((s8 >> i & 1u) && c + i < V) x[u][i] = pen.apply(x[u][i], counts[c + i]);
    }
    if (p.r.bias) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < V) x[u][i] += bias_at(p.r, bias0 + c + i);
    }
    if (mask) {
      const uint32_t m8 = bits8(mask, W, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[u][i] = (m8 >> i & 1u) ? x[u][i] : -__builtin_inff();
    }
    if constexpr (BF) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[u][i] = bf16_rne(x[u][i]);
    }
    store8<BF>(row, c, V, whole && c + 8 <= V, x[u]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float g[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (!p.greedy) {
        const Philox4 q = philox4x32_10((uint32_t)(c >> 2) + (uint32_t)j, p.k_abs,
                                        (uint32_t)p.batch_offset + (uint32_t)b, 0u, p.seed_lo, p.seed_hi);
        g[0] = gumbel2_from_word(q.x0);
        g[1] = gumbel2_from_word(q.x1);
        g[2] = gumbel2_from_word(q.x2);
        g[3] = gumbel2_from_word(q.x3);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int v = c + 4 * j + i;
        const float sc = p.greedy ? x[u][4 * j + i] : __builtin_fmaf(x[u][4 * j + i], p.kappa, g[i]);
        if (v < V) best = max_u64(best, argmax_key(sc, (uint32_t)v));
      }
    }
  }
  best = wave_max_u64_lane63(best);
  if ((tid & 63) == 63) lds_key[tid >> 6] = best;
  __syncthreads();
  if (tid == 0) {
#pragma unroll
    for (int w = 1; w < kRuleThreads / 64; ++w) best = max_u64(w == 1 ? lds_key[0] : best, lds_key[w]);
    p.partials[b * parts + part] = best;
  }
}

hipError_t launch_rule_select(const SelectParams& p, bool logits_bf16, hipStream_t s) {
  const int64_t parts = select_parts(p.V);
  if (p.B * parts > 0x7FFFFFFF) return hipErrorNotSupported;
  const bool whole = (uintptr_t)p.logits % 16 == 0 && p.V % 8 == 0;
  const dim3 grid((unsigned)(p.B * parts)), block(kRuleThreads);
  if (logits_bf16)
    hipLaunchKernelGGL(rule_select_kernel<true>, grid, block, 0, s, p, (int)parts, whole);
  else
    hipLaunchKernelGGL(rule_select_kernel<false>, grid, block, 0, s, p, (int)parts, whole);
  return hipGetLastError();
}

// One workgroup per row.  The row's table belongs to this workgroup alone, so
// the drawn token joins it without atomics; its count starts here when its
// bit was clear.
__global__ __launch_bounds__(kRuleThreads) void rule_choose_kernel(const uint64_t* __restrict__ partials,
                                                                   int64_t nparts, int64_t M, int64_t k, int64_t V,
                                                                   int64_t* __restrict__ tokens, uint32_t* seen,
                                                                   uint32_t* counts) {
  __shared__ uint64_t lds_key[kRuleThreads / 64];
  const int64_t b = blockIdx.x;
  const int tid = threadIdx.x;
  uint64_t best = 0;
  for (int64_t i = tid; i < nparts; i += kRuleThreads) best = max_u64(best, partials[b * nparts + i]);
  best = wave_max_u64_lane63(best);
  if ((tid & 63) == 63) lds_key[tid >> 6] = best;
  __syncthreads();
  if (tid == 0) {
    for (int w = 0; w < kRuleThreads / 64; ++w) best = max_u64(best, lds_key[w]);
    const uint32_t lowest = 0x007FFFFFu;  // the code of -inf: nothing was left to draw
    const int64_t t = (uint32_t)(best >> 32) > lowest ? key_index(best) : -1;
    tokens[b * M + k] = t;
    if (seen && t >= 0) {
      uint32_t* const w = seen + b * ((V + 31) / 32) + (t >> 5);
      const uint32_t bit = 1u << (t & 31);
      const bool was = (*w & bit) != 0u;
      counts[b * V + t] = was ? counts[b * V + t] + 1u : 1u;
      *w |= bit;
    }
  }
}

hipError_t launch_rule_choose(const uint64_t* partials, int64_t nparts, int64_t B, int64_t M, int64_t k, int64_t V,
                              int64_t* tokens, uint32_t* seen, uint32_t* counts, hipStream_t s) {
  if (B > 0x7FFFFFFF) return hipErrorNotSupported;
  hipLaunchKernelGGL(rule_choose_kernel, dim3((unsigned)B), dim3(kRuleThreads), 0, s, partials, nparts, M, k, V,
                     tokens, seen, counts);
  return hipGetLastError();
}

}  // namespace dspark
