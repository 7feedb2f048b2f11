// fp4_head.hip -- the vocabulary head in microscaled 4-bit floating point
// (gfx950).
//
// A block of 32 numbers x is held as codes c[i] of the fifteen values
// 0, +-1/2, +-1, +-3/2, +-2, +-3, +-4, +-6 (e2m1) and one power of two
// 2^e (e8m0), e = floor(log2 max|x|) - 2, c[i] the value nearest to x[i] / 2^e
// (ties to the even code, at most 6); the head's rows once, when its weights
// are loaded, the hidden states in the call.  The logits are
//     U[n, v] = sum_b 2^(e[n, b] + f[v, b]) sum_i c[n, b, i] h[v, b, i],
// products and sums in fp32 by the matrix cores, which take both scales.
#include <type_traits>

#include "device_common.h"
#include "fp4_head.h"

namespace dspark {

// ---------------------------------------------------------------- quantiser
namespace {
constexpr int kFp4Threads = 256;

// Biased exponent byte of a block whose largest |x| has these bits: the
// float's own less 2 (the exponent of the largest code, 6 = 1.5 * 2^2), 0 for
// what lies below, 255 where the block holds an infinity or NaN.
__device__ __forceinline__ uint32_t fp4_scale_byte(uint32_t top) {
  const uint32_t e = top >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^(byte - 127); NaN for 255.
__device__ __forceinline__ float fp4_scale(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

// Max over a quad's lanes.
__device__ __forceinline__ uint32_t quad_max_u32(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));  // quad_perm 1 0 3 2
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));  // quad_perm 2 3 0 1
  return v;
}
}  // namespace

// A lane takes 8 consecutive numbers of a row (16 bytes of bf16), a quad a
// block, 16 lanes four blocks, whose scale bytes leave as one word.  NV
// vectors a lane, a whole grid's width apart, are loaded before the first is
// used.  VEC: rows are whole aligned vectors; else numbers are loaded one by
// one.  Bound by HBM: a bf16 head of 129280 x 5120 (1.7 GB) takes 270 us, 6.2 TB/s.
template <bool BF, bool VEC, int NV>
__global__ __launch_bounds__(kFp4Threads) void fp4_quantize_kernel(Fp4QuantizeParams p, int64_t n8) {
  constexpr int NW = BF ? 1 : 2;
  const int64_t first = (int64_t)blockIdx.x * (kFp4Threads * NV) + threadIdx.x;
  const uint32_t per = (uint32_t)(p.ldc / 4);  // vectors of a row
  u32x4_t raw[NV][NW];
  uint32_t at[NV];
  int64_t row[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t i = first + j * kFp4Threads;
    row[j] = n8 <= 0xFFFFFFFFll ? (int64_t)((uint32_t)i / per) : i / per;
    at[j] = 8u * (uint32_t)(i - row[j] * per);
    const bool live = i < n8;
#pragma unroll
    for (int h = 0; h < NW; ++h) raw[j][h] = u32x4_t{0u, 0u, 0u, 0u};
    if constexpr (VEC) {
      if (live && at[j] < p.d) {
        const u32x4_t* const src = (const u32x4_t*)((const char*)p.x + (row[j] * p.d + at[j]) * (BF ? 2 : 4));
#pragma unroll
        for (int h = 0; h < NW; ++h) raw[j][h] = __builtin_nontemporal_load(src + h);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (live && at[j] + e < p.d) {
          const int64_t k = row[j] * p.d + at[j] + e;
          if constexpr (BF) raw[j][0][e >> 1] |= (uint32_t)((const uint16_t*)p.x)[k] << (16 * (e & 1));
          else raw[j][e >> 2][e & 3] = ((const uint32_t*)p.x)[k];
        }
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float x[8];
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (BF) x[e] = (e & 1) ? bf16_hi(raw[j][0][e >> 1]) : bf16_lo(raw[j][0][e >> 1]);
      else x[e] = __uint_as_float(raw[j][e >> 2][e & 3]);
      top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
    }
    const uint32_t byte = fp4_scale_byte(quad_max_u32(top));
    const float s = fp4_scale(byte);
    uint32_t c = 0;
    // v_cvt_scalef32_pk_fp4_f32: x / s to the nearest code, ties to even, at most 6
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], s, 3);
    if (byte == 255u) c = 0;
    // the bytes of the 16 lanes' four blocks, or-ed over the lanes
    uint32_t w = byte << (8 * (threadIdx.x >> 2 & 3));
    w |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x124, 0xF, 0xF, false);  // row_ror:4
    w |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x128, 0xF, 0xF, false);  // row_ror:8
    if (first + j * kFp4Threads < n8) {
      __builtin_nontemporal_store(c, (uint32_t*)(p.codes + row[j] * p.ldc + at[j] / 2));
      if ((threadIdx.x & 15) == 0) *(uint32_t*)(p.scales + row[j] * (p.ldc / 16) + at[j] / 32) = w;
    }
  }
}

// A lane takes the 8 numbers of a word of codes, as above; the same head back to
// bf16 takes 266 us, 6.3 TB/s.
template <bool BF, bool VEC, int NV>
__global__ __launch_bounds__(kFp4Threads) void fp4_dequantize_kernel(Fp4DequantizeParams p, int64_t n8) {
  const int64_t first = (int64_t)blockIdx.x * (kFp4Threads * NV) + threadIdx.x;
  const uint32_t per = (uint32_t)(p.blocks * 4);
  uint32_t c[NV], b[NV], at[NV];
  int64_t row[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t i = first + j * kFp4Threads;
    row[j] = n8 <= 0xFFFFFFFFll ? (int64_t)((uint32_t)i / per) : i / per;
    at[j] = 8u * (uint32_t)(i - row[j] * per);
    c[j] = b[j] = 0;
    if (i < n8) {
      c[j] = __builtin_nontemporal_load((const uint32_t*)p.codes + i);
      b[j] = p.scales[i >> 2];
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (first + j * kFp4Threads >= n8 || at[j] >= p.d) continue;
    const float s = fp4_scale(b[j]);
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    f32x2_t y[4];
    y[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[j], 1.0f, 0);
    y[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[j], 1.0f, 1);
    y[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[j], 1.0f, 2);
    y[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[j], 1.0f, 3);
    const int64_t k = row[j] * p.d + at[j];
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float lo = y[e][0] * s, hi = y[e][1] * s;
      if constexpr (BF) {
        o[e] = pack_bf16x2(lo, hi);
      } else {
        o[2 * e] = __float_as_uint(lo);
        o[2 * e + 1] = __float_as_uint(hi);
      }
    }
    if constexpr (VEC) {
      u32x4_t* const dst = (u32x4_t*)((char*)p.x + k * (BF ? 2 : 4));
      __builtin_nontemporal_store(u32x4_t{o[0], o[1], o[2], o[3]}, dst);
      if constexpr (!BF) __builtin_nontemporal_store(u32x4_t{o[4], o[5], o[6], o[7]}, dst + 1);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at[j] + e < p.d) {
          if constexpr (BF) ((uint16_t*)p.x)[k + e] = (uint16_t)(o[e >> 1] >> (16 * (e & 1)));
          else ((uint32_t*)p.x)[k + e] = o[e];
        }
    }
  }
}

namespace {
// Rows of a part, so that its workgroups fit one launch.
int64_t fp4_part_rows(int64_t per_row, int64_t per_group) {
  const int64_t n = kLaunchGroups * per_group / per_row;
  return n > 0 ? n : 1;
}
template <bool BF, bool VEC>
hipError_t fp4_quantize_go(const Fp4QuantizeParams& p, hipStream_t s) {
  constexpr int NV = BF ? 4 : 2;
  const int64_t per = p.ldc / 4, step = fp4_part_rows(per, kFp4Threads * NV);
  for (int64_t r = 0; r < p.rows; r += step) {
    Fp4QuantizeParams q = p;
    q.rows = p.rows - r < step ? p.rows - r : step;
    q.x = (const char*)p.x + r * p.d * (BF ? 2 : 4);
    q.codes = p.codes + r * p.ldc;
    q.scales = p.scales + r * (p.ldc / 16);
    const int64_t n8 = q.rows * per;
    hipLaunchKernelGGL((fp4_quantize_kernel<BF, VEC, NV>), dim3((unsigned)((n8 + kFp4Threads * NV - 1) / (kFp4Threads * NV))),
                       dim3(kFp4Threads), 0, s, q, n8);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <bool BF, bool VEC>
hipError_t fp4_dequantize_go(const Fp4DequantizeParams& p, hipStream_t s) {
  constexpr int NV = 4;
  const int64_t per = p.blocks * 4, step = fp4_part_rows(per, kFp4Threads * NV);
  for (int64_t r = 0; r < p.rows; r += step) {
    Fp4DequantizeParams q = p;
    q.rows = p.rows - r < step ? p.rows - r : step;
    q.x = (char*)p.x + r * p.d * (BF ? 2 : 4);
    q.codes = p.codes + r * p.blocks * 16;
    q.scales = p.scales + r * p.blocks;
    const int64_t n8 = q.rows * per;
    hipLaunchKernelGGL((fp4_dequantize_kernel<BF, VEC, NV>),
                       dim3((unsigned)((n8 + kFp4Threads * NV - 1) / (kFp4Threads * NV))), dim3(kFp4Threads), 0, s, q, n8);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
}  // namespace

hipError_t launch_fp4_quantize(const Fp4QuantizeParams& p, bool bf16, hipStream_t s) {
  if (p.d > kFp4MaxInner || p.ldc % 64 != 0 || p.ldc < 16 * fp4_blocks(p.d)) return hipErrorNotSupported;
  const bool vec = p.d % 8 == 0 && (uintptr_t)p.x % 16 == 0;
  if (bf16) return vec ? fp4_quantize_go<true, true>(p, s) : fp4_quantize_go<true, false>(p, s);
  return vec ? fp4_quantize_go<false, true>(p, s) : fp4_quantize_go<false, false>(p, s);
}

hipError_t launch_fp4_dequantize(const Fp4DequantizeParams& p, bool bf16, hipStream_t s) {
  if (p.d > kFp4MaxInner || p.blocks != fp4_blocks(p.d)) return hipErrorNotSupported;
  const bool vec = p.d % 8 == 0 && (uintptr_t)p.x % 16 == 0;
  if (bf16) return vec ? fp4_dequantize_go<true, true>(p, s) : fp4_dequantize_go<true, false>(p, s);
  return vec ? fp4_dequantize_go<false, true>(p, s) : fp4_dequantize_go<false, false>(p, s);
}

// ---------------------------------------------------------------- product
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));  // rows of the output start at any element

// c += a b by v_mfma_scale_f32_32x32x64_f8f6f4 on 4-bit codes: lane l holds
// the 32 codes of row (column) l % 32 and block l / 32, whose scale is byte S
// of sa (sb).
template <int S>
__device__ __forceinline__ f32x16_t mfma_fp4(i32x4_t a, i32x4_t b, f32x16_t c, uint32_t sa, uint32_t sb) {
  const i32x8_t a8 = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8_t b8 = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, S, (int)sa, S, (int)sb);
}

// Loads to LDS as load_lds16 and load_lds4, with a scalar offset besides the
// lanes' (which need no addition for each load then): past the buffer's end
// where their sum is.  soff is at most the buffer's size.
__device__ __forceinline__ void load_lds16_at(const BufferWords& r, uint32_t off, uint32_t soff, uint32_t lds) {
  uint32_t saved;
  __asm__ volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %4\n\ts_nop 2\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds\n\ts_mov_b32 m0, %0"
                   : "=&s"(saved) : "v"(off), "s"(r.w), "s"(soff), "s"(__builtin_amdgcn_readfirstlane(lds)) : "memory");
}
__device__ __forceinline__ void load_lds4_at(const BufferWords& r, uint32_t off, uint32_t soff, uint32_t lds) {
  uint32_t saved;
  __asm__ volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %4\n\ts_nop 2\n\tbuffer_load_dword %1, %2, %3 offen lds\n\ts_mov_b32 m0, %0"
                   : "=&s"(saved) : "v"(off), "s"(r.w), "s"(soff), "s"(__builtin_amdgcn_readfirstlane(lds)) : "memory");
}

// A workgroup of WM x WN waves owns tiles of 32 MI WM rows x 32 NJ WN
// vocabulary columns and walks them in a persistent loop; a wave holds MI x
// NJ blocks of 32 x 32 sums.  The inner dimension is cut into chunks of 128
// bytes of codes (256 numbers; half of that reads L2 at half its rate) and
// their 8 scale bytes; a chunk's rows of codes (16 bytes a lane) and of scales
// (4 bytes a lane) are loaded straight into LDS, up to STAGES chunks at a time.
// A row's eight 16-byte pieces sit at positions piece ^ (row / 2 % 8): a
// fragment read takes sixteen consecutive rows at a time, over LDS's 64 banks,
// and these fall on all of them once (216 bytes a clock and CU, against 117 at
// piece ^ (row % 8), where rows eight apart meet).  The chunk stream runs on
// across tiles.
//
// The rows of codes of x are padded with zeros to whole chunks, and scales past
// a row's blocks are read as zeros (2^-127), so that what of the head's next
// row stands in a last chunk counts nothing, NaN scales included.
//
// AHEAD (tiles bound by the matrix cores): fragments are read while earlier
// products run, and the hand-over from chunk to chunk (its loads one by one
// between products, then wait, barrier and first reads) runs behind the chunk's
// last two steps; with all of it behind the last one, 2560 rows took 968 us
// instead of 940.  The sums are pinned after
// each step, or the compiler would move all of a chunk's products past the wait
// for the next one's loads (at 2560 rows 9% of the time).
// Otherwise (tiles bound by the head's stream) all of a chunk's fragments are
// read at once, so that their latency is paid once a chunk.
template <int MI, int NJ, int WM, int WN, int STAGES, bool AHEAD, bool OBF>
__global__ __launch_bounds__(64 * WM * WN) void fp4_head_kernel(Fp4HeadParams p, int row_tiles, int tiles) {
  constexpr int NW = WM * WN;
  constexpr int BM = 32 * MI * WM, BN = 32 * NJ * WN, BK = (int)kFp4K, SB = BK / 16;
  constexpr int CODES = (BM + BN) * BK, STAGE = CODES + (BM + BN) * SB;
  // load instructions of a chunk per wave: of 8 rows of codes, and of 32 rows of scales
  constexpr int PA = BM / 8 / NW, PB = BN / 8 / NW, SI = (BM + BN) / 32, PS = (SI + NW - 1) / NW, PER = PA + PB + PS;
  static_assert(BM / 8 % NW == 0 && BN / 8 % NW == 0, "whole load instructions per wave");
  static_assert((STAGES - 1) * PER < 64, "wait count");
  // a wave's part of the output on its way to memory: ER rows x 32 NJ columns
  constexpr int STORES = MI * NJ * (OBF ? 2 : 4);  // instructions for a wave's part of a whole tile
  static_assert(!AHEAD || (STAGES == 2 && PER < 63), "the hand-over's wait counts");
  constexpr int OS = OBF ? 2 : 4, ER = OBF ? 16 : 8, EROW = 32 * NJ * OS, EBYTES = ER * EROW;
  __shared__ __attribute__((aligned(16))) unsigned char lds[STAGES * STAGE + NW * EBYTES];

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int wm = wave / WN, wn = wave % WN;
  const int C = (int)(p.ldx / BK);
  const uint32_t ldx = (uint32_t)p.ldx, ldw = 16u * (uint32_t)p.blocks, lxs = ldx / 16, lws = (uint32_t)p.blocks;

  // tile i of this workgroup: neighbouring workgroups of one XCD (every
  // eighth) take neighbouring tiles, rows first, so that they share the rows
  // of the head in that XCD's L2
  const int G = (int)gridDim.x;
  const int first = G % 8 == 0 ? ((int)blockIdx.x % 8) * (G / 8) + (int)blockIdx.x / 8 : (int)blockIdx.x;
  const int my = first < tiles ? (tiles - 1 - first) / G + 1 : 0;

  // ---- the load stream
  int lt = 0, lc = 0;  // tile (of mine) and chunk
  BufferWords ba, bb, sa, sb;
  auto bind = [&](int t) __attribute__((always_inline)) {
    const int tile = first + t * G;
    const int64_t r0 = (int64_t)(tile % row_tiles) * BM, v0 = (int64_t)(tile / row_tiles) * BN;
    const uint32_t nr = (uint32_t)(p.rows - r0 < BM ? p.rows - r0 : BM), nv = (uint32_t)(p.V - v0 < BN ? p.V - v0 : BN);
    ba = buffer_words(p.xc + r0 * ldx, nr * ldx);
    bb = buffer_words(p.wc + v0 * ldw, nv * ldw);
    sa = buffer_words(p.xs + r0 * lxs, nr * lxs);
    sb = buffer_words(p.ws + v0 * lws, nv * lws);
  };
  // load instruction j of this wave fills rows 8 (wave + j NW) .. + 7, lane l
  // the position l % 8 of row l / 8 (which holds piece l % 8 ^ row / 2 % 8); the
  // scales' fill rows 32 i .. + 31 of x, then of the head, lane l word l % 2 of
  // row l / 2 (every wave issues PS of them, the last one over again)
  const uint32_t row8 = 8u * (uint32_t)wave + (uint32_t)(lane >> 3);
  const uint32_t q16 = 16u * ((uint32_t)(lane & 7) ^ (row8 >> 1 & 7));
  static_assert(NW % 2 == 0, "a lane's swizzle is the same for all its rows");
  uint32_t offa[PA], offb[PB], offs[PS];
#pragma unroll
  for (int j = 0; j < PA; ++j) offa[j] = (row8 + (uint32_t)(8 * NW * j)) * ldx + q16;
#pragma unroll
  for (int j = 0; j < PB; ++j) offb[j] = (row8 + (uint32_t)(8 * NW * j)) * ldw + q16;
  auto scale_rows = [&](int j) __attribute__((always_inline)) { return wave + NW * j < SI ? wave + NW * j : SI - 1; };
#pragma unroll
  for (int j = 0; j < PS; ++j) {
    const int i = scale_rows(j);
    const bool x = NW * (j + 1) <= BM / 32 || (NW * j < BM / 32 && i < BM / 32);
    offs[j] = (32u * (uint32_t)(x ? i : i - BM / 32) + (uint32_t)(lane >> 1)) * (x ? lxs : lws) + 4u * (uint32_t)(lane & 1);
  }
  auto load = [&](int g, int q) __attribute__((always_inline)) {  // load q of chunk g of the stream
    const uint32_t k0 = (uint32_t)lc * BK, stage = lds_address(&lds[(uint32_t)(g % STAGES) * STAGE]);
    if (q < PA) {
      load_lds16_at(ba, offa[q < PA ? q : 0], k0, stage + 1024u * (uint32_t)(wave + NW * q));
    } else if (q < PA + PB) {
      const int j = q - PA;
      load_lds16_at(bb, offb[j < PB ? j : 0], k0, stage + BM * BK + 1024u * (uint32_t)(wave + NW * j));
    } else {
      const int j = q - PA - PB, i = scale_rows(j);
      const bool x = NW * (j + 1) <= BM / 32 || (NW * j < BM / 32 && i < BM / 32);  // the compiler knows it for most j
      const uint32_t k = (uint32_t)lc * SB;
      load_lds4_at(x ? sa : sb, k + 4u * (uint32_t)(lane & 1) < (x ? lxs : lws) ? offs[j < PS ? j : 0] : kBufferOob, k,
                   stage + CODES + 256u * (uint32_t)i);
    }
  };
  auto next = [&]() __attribute__((always_inline)) {  // on to the stream's next chunk
    if (lt < my && ++lc == C) {
      lc = 0;
      if (++lt < my) bind(lt);
      else ba = bb = sa = sb = buffer_words(p.xc, 0);  // the loads past the last chunk bring zeros
    }
  };
  auto issue = [&](int g) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < PER; ++q) load(g, q);
    next();
  };

  // ---- the products: fragments of the wave's MI x NJ blocks for one matrix
  // instruction each, and a chunk's scales of its rows, the four of the lane's
  // half (blocks of even or odd number) in one word
  constexpr int S = BK / 32;
  struct Frags {
    i32x4_t a[MI], b[NJ];
  };
  struct Scales {
    uint32_t a[MI], b[NJ];
  };
  auto read = [&](int g, int s, Frags& f) __attribute__((always_inline)) {  // step s of chunk g
    const int piece = 16 * ((2 * s + (lane >> 5)) ^ (lane >> 1 & 7)) + (lane & 31) * BK;
    const unsigned char* const x = &lds[(g % STAGES) * STAGE + piece];
    const unsigned char* const h = x + BM * BK;
#pragma unroll
    for (int i = 0; i < MI; ++i) f.a[i] = *(const i32x4_t*)(x + 32 * (MI * wm + i) * BK);
#pragma unroll
    for (int j = 0; j < NJ; ++j) f.b[j] = *(const i32x4_t*)(h + 32 * (NJ * wn + j) * BK);
  };
  const uint32_t pick = lane >> 5 ? 0x07050301u : 0x06040200u;
  auto read_scales = [&](int g, Scales& f) __attribute__((always_inline)) {
    const unsigned char* const x = &lds[(g % STAGES) * STAGE + CODES + (lane & 31) * SB];
    const unsigned char* const h = x + BM * SB;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const uint64_t w = *(const uint64_t*)(x + 32 * (MI * wm + i) * SB);
      f.a[i] = __builtin_amdgcn_perm((uint32_t)(w >> 32), (uint32_t)w, pick);
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const uint64_t w = *(const uint64_t*)(h + 32 * (NJ * wn + j) * SB);
      f.b[j] = __builtin_amdgcn_perm((uint32_t)(w >> 32), (uint32_t)w, pick);
    }
  };
  f32x16_t acc[MI][NJ];
  // product q of step s
  auto product = [&](auto s, int q, const Frags& f, const Scales& sc) __attribute__((always_inline)) {
    const int i = q / NJ, j = q % NJ;
    acc[i][j] = mfma_fp4<decltype(s)::value>(f.a[i], f.b[j], acc[i][j], sc.a[i], sc.b[j]);
    if constexpr (AHEAD) __asm__ volatile("" : "+a"(acc[i][j]));  // no instruction: the sum stays in its place
  };
  auto multiply = [&](auto s, const Frags& f, const Scales& sc) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < MI * NJ; ++q) product(s, q, f, sc);
    if constexpr (AHEAD) __builtin_amdgcn_sched_barrier(0);
  };
  using std::integral_constant;
  constexpr integral_constant<int, 0> s0{};
  constexpr integral_constant<int, 1> s1{};
  constexpr integral_constant<int, 2> s2{};
  constexpr integral_constant<int, 3> s3{};
  static_assert(S == 4, "steps of a chunk");

  if (my == 0) return;
  bind(0);
#pragma unroll
  for (int g = 0; g < STAGES - (AHEAD ? 0 : 1); ++g) issue(g);
  Frags f[AHEAD ? 3 : S];
  Scales sc, sn;
  if constexpr (AHEAD) {
    wait_vmcnt<(STAGES - 1) * PER>();
    lds_barrier();
    read(0, 0, f[0]);
    read_scales(0, sc);
  }
  int g = 0, landed = 0;  // landed: steps whose chunk is known to have arrived
  bool stored = false;    // the wave's part of the last tile was whole
  for (int t = 0; t < my; ++t) {
    const int tile = first + t * G;
    const int64_t r0 = (int64_t)(tile % row_tiles) * BM + 32 * MI * wm;
    const int64_t v0 = (int64_t)(tile / row_tiles) * BN + 32 * NJ * wn;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    for (int c = 0; c < C; ++c, ++g) {
      if constexpr (AHEAD) {
        // Fragments are read up to two steps ahead.  When step 3's have come to
        // every wave, the chunk's stage takes the loads of chunk g + STAGES, one
        // by one between step 2's products; the next chunk's have landed for
        // every wave before step 3, behind whose products its first fragments
        // and scales are read.
        read(g, 1, f[1]);
        read(g, 2, f[2]);
        multiply(s0, f[0], sc);
        read(g, 3, f[0]);
        multiply(s1, f[1], sc);
        lds_barrier();
#pragma unroll
        for (int q = 0; q < MI * NJ; ++q) {
          product(s2, q, f[2], sc);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int l = q * PER / (MI * NJ); l < (q + 1) * PER / (MI * NJ); ++l) load(g + STAGES, l);
          __builtin_amdgcn_sched_barrier(0);
        }
        // (Loads and stores are counted in the order of their issue: the next
        // chunk's are older than these, and than the last tile's stores, which
        // may go on.)
        if (c == 0 && stored) wait_vmcnt<(STORES + PER < 63 ? STORES + PER : 63)>();
        else wait_vmcnt<PER>();
        lds_barrier();
        read(g + 1, 0, f[1]);
        read_scales(g + 1, sn);
        __builtin_amdgcn_sched_barrier(0);
        multiply(s3, f[0], sc);
        f[0] = f[1];
        next();
        sc = sn;
      } else {
        // chunk g has landed for every wave, and every wave has read chunk g - 1
        if (landed > 0) --landed;
        else wait_vmcnt<(STAGES - 2) * PER>();
        lds_barrier();
        issue(g + STAGES - 1);
        read_scales(g, sc);
#pragma unroll
        for (int s = 0; s < S; ++s) read(g, s, f[s]);
        multiply(s0, f[0], sc);
        multiply(s1, f[1], sc);
        multiply(s2, f[2], sc);
        multiply(s3, f[3], sc);
      }
    }
    if constexpr (!AHEAD) {
      // the chunks on their way (the last was issued a step ago), so that the
      // next steps need not wait for the stores
      wait_vmcnt<0>();
      landed = STAGES - 1;
    }
    // Lane l holds column l % 32 of rows 8 (e / 4) + 4 (l / 32) + e % 4 of each
    // block, which as they are would leave in stores of one element a lane.  So
    // ER rows at a time go through the wave's own LDS, in 16-byte pieces, those
    // of every other four rows moved by half a row so that both halves of the
    // wave write to different banks, and leave in whole pieces of consecutive
    // columns.
    unsigned char* const mine = &lds[STAGES * STAGE + wave * EBYTES];
    stored = r0 + 32 * MI <= p.rows && v0 + 32 * NJ <= p.V;  // no lane of the stores below is left out
    constexpr int PIECES = EROW / 16, HALF = PIECES / 2;  // of a row
    constexpr int SETS = ER / 8;                          // groups of 8 rows in an exchange
    auto turned = [](int q, int half) __attribute__((always_inline)) {
      const int r = q + HALF * half;
      return r < PIECES ? r : r - PIECES;
    };
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int x = 0; x < 4 / SETS; ++x) {
        const int64_t rb = r0 + 32 * i + ER * x;  // first row of the exchange
        if (rb >= p.rows) continue;
        // Lanes' addresses are computed anew each time: kept over the products
        // they go to scratch, and each reload waits for all stores before it.
        int l = lane;
        __asm__ volatile("" : "+v"(l));
        if constexpr (AHEAD) {
          // nor are sums that a later exchange takes read yet
#pragma unroll
          for (int k = i; k < MI; ++k)
#pragma unroll
            for (int j = 0; j < NJ; ++j) __asm__ volatile("" : "+a"(acc[k][j]));
        }
#pragma unroll
        for (int u = 0; u < SETS; ++u) {
          const int lr = 8 * u + 4 * (l >> 5);  // first of the lane's four rows
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              const float y = acc[i][j][4 * (SETS * x + u) + e];
              const int byte = (32 * j + (l & 31)) * OS;
              unsigned char* const at = mine + (lr + e) * EROW + 16 * turned(byte >> 4, l >> 5) + (byte & 15);
              if constexpr (OBF) *(uint16_t*)at = (uint16_t)(pack_bf16x2(y, 0.0f) & 0xFFFFu);
              else *(float*)at = y;
            }
        }
#pragma unroll
        for (int h = 0; h < ER * PIECES / 64; ++h) {
          const int pc = l + 64 * h, lr = pc / PIECES, q = pc % PIECES;
          const u32x4_t w = *(const u32x4_t*)(mine + lr * EROW + 16 * turned(q, lr >> 2 & 1));
          const int64_t n = rb + lr, v = v0 + q * (16 / OS);
          unsigned char* const dst = (unsigned char*)p.out + (rb * p.V + v0) * OS + ((int64_t)lr * p.V + q * (16 / OS)) * OS;
          if (stored || (n < p.rows && v + 16 / OS <= p.V)) {
            __builtin_nontemporal_store(w, (u32x4_any_t*)dst);
          } else if (n < p.rows && v < p.V) {
            for (int e = 0; e < (int)(p.V - v); ++e) {
              if constexpr (OBF) ((uint16_t*)dst)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
              else ((uint32_t*)dst)[e] = w[e];
            }
          }
        }
      }
  }
  wait_vmcnt<0>();
}

namespace {
template <int MI, int NJ, int WM, int WN, int STAGES, bool AHEAD>
hipError_t head_go(const Fp4HeadParams& p, bool obf, int groups, hipStream_t s) {
  constexpr int BM = 32 * MI * WM, BN = 32 * NJ * WN;
  const int64_t rt = (p.rows + BM - 1) / BM, tiles = rt * ((p.V + BN - 1) / BN);
  if (tiles > 0x3FFFFFFF || rt > 0x3FFFFFFF) return hipErrorNotSupported;
  // persistent: a workgroup's chunk count is an int
  if ((tiles / groups + 1) * (p.ldx / kFp4K) > 0x3FFFFFFF) return hipErrorNotSupported;
  const dim3 grid((unsigned)(tiles < groups ? tiles : groups)), block(64 * WM * WN);
  if (obf)
    hipLaunchKernelGGL((fp4_head_kernel<MI, NJ, WM, WN, STAGES, AHEAD, true>), grid, block, 0, s, p, (int)rt, (int)tiles);
  else
    hipLaunchKernelGGL((fp4_head_kernel<MI, NJ, WM, WN, STAGES, AHEAD, false>), grid, block, 0, s, p, (int)rt, (int)tiles);
  return hipGetLastError();
}
}  // namespace

// The forms of the kernel, and what their tiles over the CUs take: the first
// round of them and every further one (us at d = 5120, the one hidden size at
// which they were timed against each other).  The form with the shortest sum is
// taken.  Kernel times at V = 129280, in us, bf16 logits from 128 rows on: 1 row
// 70 (32x128), 68 (32x256); 64 rows 117 (32x128), 95 (64x128), 81 (64x256), 102
// (128x256); 128 rows 137 (64x256), 90 (128x256), 105 (192x256), 101 (256x256); 256
// rows 152 (128x256), 109 (256x256), 134 (320x192); 320 rows 197 (128x256), 171
// (192x256), 175 (256x256), 152 (320x128), 142 (320x192); 640 rows 326, 309, 273,
// 281, 257; 2560 rows 1239, 1053, 934, 1103, 962.  37 rows of 2056 at V = 32003:
// 13.5 (32x128), 9.1 (64x128), 12.8 (64x256).
namespace {
struct Form {
  int bm, bn;
  float first, more;
};
constexpr Form kForms[] = {{32, 128, 17.5f, 17.5f}, {64, 128, 24.0f, 24.0f},  {64, 256, 40.0f, 40.0f},  {128, 256, 62.0f, 31.0f},
                           {192, 256, 69.0f, 37.0f}, {256, 256, 56.0f, 46.5f}, {320, 128, 42.0f, 35.0f}, {320, 192, 52.0f, 44.0f}};
int pick_form(int64_t rows, int64_t V, int num_cus) {
  int best = 0;
  double least = 0.0;
  for (int i = 0; i < (int)(sizeof(kForms) / sizeof(kForms[0])); ++i) {
    const Form& f = kForms[i];
    const int64_t tiles = ((rows + f.bm - 1) / f.bm) * ((V + f.bn - 1) / f.bn);
    const double cost = f.first + (double)((tiles + num_cus - 1) / num_cus - 1) * f.more;
    if (i == 0 || cost < least) {
      best = i;
      least = cost;
    }
  }
  return best;
}
}  // namespace

hipError_t launch_fp4_head(const Fp4HeadParams& p, bool out_bf16, int num_cus, hipStream_t s) {
  if (num_cus < 1 || p.ldx % kFp4K != 0 || p.ldx < 16 * p.blocks || p.blocks % 4 != 0 || 32 * p.blocks > kFp4MaxInner)
    return hipErrorNotSupported;
  switch (pick_form(p.rows, p.V, num_cus)) {
    case 0: return head_go<1, 1, 1, 4, 4, false>(p, out_bf16, num_cus, s);
    case 1: return head_go<1, 1, 2, 4, 3, false>(p, out_bf16, num_cus, s);
    case 2: return head_go<1, 2, 2, 4, 3, false>(p, out_bf16, num_cus, s);
    case 3: return head_go<2, 4, 2, 2, 2, true>(p, out_bf16, num_cus, s);
    case 4: return head_go<3, 4, 2, 2, 2, true>(p, out_bf16, num_cus, s);
    case 5: return head_go<4, 4, 2, 2, 2, true>(p, out_bf16, num_cus, s);
    case 6: return head_go<5, 2, 2, 2, 2, true>(p, out_bf16, num_cus, s);
    default: return head_go<5, 3, 2, 2, 2, true>(p, out_bf16, num_cus, s);
  }
}

}  // namespace dspark
