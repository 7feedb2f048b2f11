// int8_head.hip -- the vocabulary head in 8-bit integers (gfx950).
//
// A row x of hidden states is held as q[i] = rint(x[i] / s), s = max|x| / 127,
// and every vocabulary row of the head the same way (once, when its weights
// are loaded), so that
//     U[n, v] = (s[n] * t[v]) * sum_i q[n, i] h[v, i]
// where the sum of products is exact in 32-bit integers: only the scales and
// the conversion of the sum round.
#include "device_common.h"
#include "int8_head.h"

namespace dspark {

// ---------------------------------------------------------------- quantiser
namespace {

constexpr int kQuantThreads = 256;

// Max of the bit patterns of |x| over a row: as integers they order like the
// values, with inf above every number and NaN above inf, so a row that holds
// either shows it in its scale.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The scale of a row, and its integers: zero where the scale is zero (a row
// of zeros, or of numbers so small that max / 127 is) or not a number.
__device__ __forceinline__ float row_scale(uint32_t top) { return __uint_as_float(top) / 127.0f; }
__device__ __forceinline__ uint32_t quantize1(float x, float s, bool ok) {
  const float q = ok ? __builtin_rintf(x / s) : 0.0f;
  return (uint32_t)(int)fminf(fmaxf(q, -127.0f), 127.0f) & 0xFFu;
}
__device__ __forceinline__ bool usable(float s) { return s > 0.0f && s < __builtin_inff(); }

}  // namespace

// LANES threads a row (64 or 256), NV vectors of 8 elements a thread held in
// registers: x is read once.  Bound by HBM.
template <bool BF, int LANES, int NV>
__global__ __launch_bounds__(kQuantThreads) void quantize_rows_kernel(QuantizeParams p) {
  __shared__ uint32_t lds_top[kQuantThreads / 64];
  const int tid = threadIdx.x;
  const int64_t row = (int64_t)blockIdx.x * (kQuantThreads / LANES) + tid / LANES;
  const int t = tid % LANES;
  const bool live = row < p.rows;
  const int64_t d8 = p.d / 8, q8 = p.ldq / 8;
  const u32x4_t* const src = (const u32x4_t*)((const char*)p.x + (live ? row : 0) * p.d * (BF ? 2 : 4));
  float x[NV][8];
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t i = t + (int64_t)j * LANES;
    u32x4_t a = {0u, 0u, 0u, 0u}, b = {0u, 0u, 0u, 0u};
    if (live && i < d8) {
      a = __builtin_nontemporal_load(src + (BF ? i : 2 * i));
      if constexpr (!BF) b = __builtin_nontemporal_load(src + 2 * i + 1);
    }
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (BF) x[j][e] = (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
      else x[j][e] = __uint_as_float(w[e]);
      top = max(top, abs_bits(x[j][e]));
    }
  }
  top = (uint32_t)__builtin_amdgcn_readlane((int)wave_max_u32_to_lane63(top), 63);
  if constexpr (LANES == kQuantThreads) {
    if ((tid & 63) == 0) lds_top[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQuantThreads / 64; ++w) top = max(top, lds_top[w]);
  }
  if (!live) return;
  const float s = row_scale(top);
  const bool ok = usable(s);
  uint64_t* const dst = (uint64_t*)(p.q + row * p.ldq);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t i = t + (int64_t)j * LANES;
    if (i >= q8) break;
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo |= quantize1(x[j][e], s, ok) << (8 * e);
      hi |= quantize1(x[j][4 + e], s, ok) << (8 * e);
    }
    dst[i] = ((uint64_t)hi << 32) | lo;  // zeros past d8: the padding
  }
  if (t == 0) p.scale[row] = s;
}

// Any d, alignment and length: a workgroup a row, read twice (the second time
// from L2).
template <bool BF>
__global__ __launch_bounds__(kQuantThreads) void quantize_rows_any_kernel(QuantizeParams p) {
  __shared__ uint32_t lds_top[kQuantThreads / 64];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const char* const src = (const char*)p.x + row * p.d * (BF ? 2 : 4);
  auto at = [&](int64_t i) __attribute__((always_inline)) {
    return BF ? bf16_lo(((const uint16_t*)src)[i]) : ((const float*)src)[i];
  };
  uint32_t top = 0;
  for (int64_t i = tid; i < p.d; i += kQuantThreads) top = max(top, abs_bits(at(i)));
  top = (uint32_t)__builtin_amdgcn_readlane((int)wave_max_u32_to_lane63(top), 63);
  if ((tid & 63) == 0) lds_top[tid >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQuantThreads / 64; ++w) top = max(top, lds_top[w]);
  const float s = row_scale(top);
  const bool ok = usable(s);
  for (int64_t i = tid; i < p.ldq; i += kQuantThreads)
    p.q[row * p.ldq + i] = (int8_t)(i < p.d ? quantize1(at(i), s, ok) : 0u);
  if (tid == 0) p.scale[row] = s;
}

namespace {
template <bool BF, int LANES, int NV>
hipError_t quantize_go(const QuantizeParams& p, hipStream_t s) {
  constexpr int per = kQuantThreads / LANES;
  hipLaunchKernelGGL((quantize_rows_kernel<BF, LANES, NV>), dim3((unsigned)((p.rows + per - 1) / per)),
                     dim3(kQuantThreads), 0, s, p);
  return hipGetLastError();
}
template <bool BF>
hipError_t quantize_pick(const QuantizeParams& p, hipStream_t s) {
  const bool vec = p.d % 8 == 0 && p.ldq % 8 == 0 && (uintptr_t)p.x % 16 == 0 && (uintptr_t)p.q % 8 == 0;
  if (vec && p.ldq <= 512) return quantize_go<BF, 64, 1>(p, s);
  if (vec && p.ldq <= 2048) return quantize_go<BF, 64, 4>(p, s);
  if (vec && p.ldq <= 4096) return quantize_go<BF, 256, 2>(p, s);
  if (vec && p.ldq <= 8192) return quantize_go<BF, 256, 4>(p, s);
  hipLaunchKernelGGL(quantize_rows_any_kernel<BF>, dim3((unsigned)p.rows), dim3(kQuantThreads), 0, s, p);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_quantize_rows(const QuantizeParams& p, bool bf16, hipStream_t s) {
  if (p.rows > 0x7FFFFFFF) return hipErrorNotSupported;
  return bf16 ? quantize_pick<true>(p, s) : quantize_pick<false>(p, s);
}

// ---------------------------------------------------------------- product
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

// A workgroup of WM x WN waves owns tiles of 32 MI WM rows x 32 NJ WN
// vocabulary columns and walks them in a persistent loop; a wave holds MI x
// NJ blocks of 32 x 32 sums.  The inner dimension is cut into chunks of 128
// bytes; a chunk's rows of q and of the head are loaded straight into LDS
// (16 bytes a lane, no registers), STAGES - 1 chunks ahead of their use.  A
// row's eight 16-byte pieces sit at positions piece ^ (row % 8), so that the
// fragment reads of eight consecutive rows fall on different banks.  The chunk
// stream runs on across tiles.
//
// v_mfma_i32_32x32x32_i8: rows of q on M, vocabulary columns on N, so that a
// store instruction writes 32 consecutive columns of two rows, whatever V's
// parity.
//
// DIRECT needs rows of the head in whole 16-byte pieces; otherwise its pieces
// go through registers by unaligned loads.
template <int MI, int NJ, int WM, int WN, int STAGES, bool DIRECT, bool OBF>
__global__ __launch_bounds__(64 * WM * WN) void int8_head_kernel(Int8HeadParams p, int row_tiles, int tiles) {
  constexpr int NW = WM * WN, THREADS = 64 * NW;
  constexpr int BM = 32 * MI * WM, BN = 32 * NJ * WN, BK = (int)kInt8K;
  constexpr int STAGE = (BM + BN) * BK;
  constexpr int IA = BM / 8, IB = DIRECT ? BN / 8 : 0;   // load instructions of a chunk, 8 rows each
  constexpr int PER = (IA + IB + NW - 1) / NW;           // per wave
  constexpr int REGS = DIRECT ? 1 : BN * 8 / THREADS;    // pieces of the head a thread moves itself
  static_assert(DIRECT || STAGES == 2, "register pieces are one chunk ahead");
  static_assert((STAGES - 2) * PER < 64, "wait count");
  constexpr int JUNK = (IA + IB) % NW ? 1024 : 0;        // where loads without a place go
  __shared__ __attribute__((aligned(16))) unsigned char lds[STAGES * STAGE + JUNK];

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int wm = wave / WN, wn = wave % WN;
  const int C = (int)(p.ldx / BK);

  // tile i of this workgroup: neighbouring workgroups of one XCD (every
  // eighth) take neighbouring tiles, rows first, so that they share the rows
  // of the head in that XCD's L2
  const int G = (int)gridDim.x;
  const int first = G % 8 == 0 ? ((int)blockIdx.x % 8) * (G / 8) + (int)blockIdx.x / 8 : (int)blockIdx.x;
  const int my = first < tiles ? (tiles - 1 - first) / G + 1 : 0;
  const int total = my * C;

  // the load stream
  int lt = 0, lc = 0;  // tile (of mine) and chunk
  BufferWords ba, bb;
  int64_t lv0 = 0;
  auto bind = [&](int t) __attribute__((always_inline)) {
    const int tile = first + t * G;
    const int64_t r0 = (int64_t)(tile % row_tiles) * BM, v0 = (int64_t)(tile / row_tiles) * BN;
    const int64_t nr = p.rows - r0 < BM ? p.rows - r0 : BM, nv = p.V - v0 < BN ? p.V - v0 : BN;
    ba = buffer_words(p.xq + r0 * p.ldx, (uint32_t)(nr * p.ldx));
    if constexpr (DIRECT) bb = buffer_words(p.wq + v0 * p.d, (uint32_t)(nv * p.d));
    lv0 = v0;
  };
  const uint32_t q16 = 16u * (uint32_t)((lane & 7) ^ (lane >> 3));  // the piece this lane's position holds
  u32x4_t held[REGS];
  auto issue = [&](int g) __attribute__((always_inline)) {  // chunk g of the stream, in order
    const bool live = g < total;
    const uint32_t k0 = (uint32_t)lc * BK + q16;
    const uint32_t stage = lds_address(&lds[(uint32_t)(g % STAGES) * STAGE]);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = wave + j * NW;  // uniform over the wave
      if (i < IA) {
        const uint32_t off = live ? (uint32_t)(8 * i + (lane >> 3)) * (uint32_t)p.ldx + k0 : kBufferOob;
        load_lds16(ba, off, stage + (uint32_t)i * 1024u);
      } else if (i < IA + IB) {
        const uint32_t off = live ? (uint32_t)(8 * (i - IA) + (lane >> 3)) * (uint32_t)p.d + k0 : kBufferOob;
        load_lds16(bb, off, stage + (uint32_t)i * 1024u);
      } else {
        load_lds16(ba, kBufferOob, lds_address(&lds[STAGES * STAGE]));
      }
    }
    if constexpr (!DIRECT) {
#pragma unroll
      for (int j = 0; j < REGS; ++j) {
        const int pc = tid + j * THREADS;
        const int64_t v = lv0 + (pc >> 3), k = (int64_t)lc * BK + 16 * (pc & 7);
        u32x4_t w = {0u, 0u, 0u, 0u};
        if (live && v < p.V && k < p.d) {
          const int8_t* const src = p.wq + v * p.d + k;
          if (k + 16 <= p.d) {
            __builtin_memcpy(&w, src, 16);
          } else {
            uint32_t b[4] = {0u, 0u, 0u, 0u};
            for (int e = 0; e < (int)(p.d - k); ++e) b[e >> 2] |= (uint32_t)(uint8_t)src[e] << (8 * (e & 3));
            w = u32x4_t{b[0], b[1], b[2], b[3]};
          }
        }
        held[j] = w;
      }
    }
    if (++lc == C) {
      lc = 0;
      if (++lt < my) bind(lt);
    }
  };
  auto put = [&](int g) __attribute__((always_inline)) {  // the held pieces, into chunk g's stage
    if constexpr (!DIRECT) {
#pragma unroll
      for (int j = 0; j < REGS; ++j) {
        const int pc = tid + j * THREADS, row = pc >> 3;
        *(u32x4_t*)&lds[(g % STAGES) * STAGE + (BM + row) * BK + 16 * ((pc & 7) ^ (row & 7))] = held[j];
      }
    }
  };

  if (my == 0) return;
  bind(0);
#pragma unroll
  for (int g = 0; g < STAGES - 1; ++g) issue(g);
  if constexpr (!DIRECT) put(0);

  i32x16_t acc[MI][NJ];
  int g = 0, landed = 0;  // steps whose chunk is known to have landed
  for (int t = 0; t < my; ++t) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
    for (int c = 0; c < C; ++c, ++g) {
      // chunk g has landed for every wave, and every wave has read chunk g - 1
      if (landed > 0) --landed;
      else wait_vmcnt<(STAGES - 2) * PER>();
      lds_barrier();
      issue(g + STAGES - 1);
      const unsigned char* const sa = &lds[(g % STAGES) * STAGE + (32 * MI * wm + (lane & 31)) * BK];
      const unsigned char* const sb = &lds[(g % STAGES) * STAGE + (BM + 32 * NJ * wn + (lane & 31)) * BK];
#pragma unroll
      for (int s = 0; s < BK / 32; ++s) {
        const int at = 16 * ((2 * s + (lane >> 5)) ^ (lane & 7));
        i32x4_t fa[MI], fb[NJ];
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[i] = *(const i32x4_t*)(sa + i * 32 * BK + at);
#pragma unroll
        for (int j = 0; j < NJ; ++j) fb[j] = *(const i32x4_t*)(sb + j * 32 * BK + at);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[i], fb[j], acc[i][j], 0, 0, 0);
      }
      if constexpr (!DIRECT) put(g + 1);
    }
    // The counted waits above hold for loads alone, so every chunk on its way
    // is waited for before the stores go out (the last was issued a step ago).
    wait_vmcnt<0>();
    landed = STAGES - 1;
    // the tile's sums times its scales: lane l holds column l % 32 of rows
    // 8 (e / 4) + 4 (l / 32) + e % 4 of each block
    const int tile = first + t * G;
    const int64_t r0 = (int64_t)(tile % row_tiles) * BM + 32 * MI * wm + 4 * (lane >> 5);
    const int64_t v0 = (int64_t)(tile / row_tiles) * BN + 32 * NJ * wn + (lane & 31);
    float wsc[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) wsc[j] = v0 + 32 * j < p.V ? p.ws[v0 + 32 * j] : 0.0f;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        const int64_t rb = r0 + 32 * i + 8 * e4;
        if (rb >= p.rows) continue;
        const f32x4_t xsc = *(const f32x4_t*)(p.xs + rb);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t n = rb + e;
          if (n >= p.rows) continue;
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const int64_t v = v0 + 32 * j;
            const float y = (xsc[e] * wsc[j]) * (float)acc[i][j][4 * e4 + e];
            if (v < p.V) {
              if constexpr (OBF)
                __builtin_nontemporal_store((uint16_t)(pack_bf16x2(y, 0.0f) & 0xFFFFu), (uint16_t*)p.out + n * p.V + v);
              else
                __builtin_nontemporal_store(y, (float*)p.out + n * p.V + v);
            }
          }
        }
      }
  }
  wait_vmcnt<0>();
}

namespace {
template <int MI, int NJ, int WM, int WN, int STAGES, bool DIRECT>
hipError_t head_go(const Int8HeadParams& p, bool obf, int groups, hipStream_t s) {
  constexpr int BM = 32 * MI * WM, BN = 32 * NJ * WN;
  const int64_t rt = (p.rows + BM - 1) / BM, tiles = rt * ((p.V + BN - 1) / BN);
  if (tiles > 0x3FFFFFFF || rt > 0x3FFFFFFF) return hipErrorNotSupported;
  // persistent: a workgroup's chunk count is an int
  if ((tiles / groups + 1) * (p.ldx / kInt8K) > 0x3FFFFFFF) return hipErrorNotSupported;
  const dim3 grid((unsigned)(tiles < groups ? tiles : groups)), block(64 * WM * WN);
  if (obf)
    hipLaunchKernelGGL((int8_head_kernel<MI, NJ, WM, WN, STAGES, DIRECT, true>), grid, block, 0, s, p, (int)rt, (int)tiles);
  else
    hipLaunchKernelGGL((int8_head_kernel<MI, NJ, WM, WN, STAGES, DIRECT, false>), grid, block, 0, s, p, (int)rt, (int)tiles);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_int8_head(const Int8HeadParams& p, bool out_bf16, int num_cus, hipStream_t s) {
  if (num_cus < 1 || p.d > kInt8MaxInner || p.ldx % kInt8K != 0 || p.ldx < p.d) return hipErrorNotSupported;
  const bool direct = p.d % 16 == 0 && (uintptr_t)p.wq % 16 == 0;
  if (!direct) return head_go<2, 1, 1, 4, 2, false>(p, out_bf16, 3 * num_cus, s);
  if (p.rows <= 32) return head_go<1, 1, 1, 4, 4, true>(p, out_bf16, num_cus, s);
  if (p.rows <= 64) return head_go<2, 1, 1, 4, 4, true>(p, out_bf16, num_cus, s);
  if (p.rows <= 128) return head_go<2, 2, 2, 4, 3, true>(p, out_bf16, num_cus, s);
  return head_go<4, 2, 2, 4, 2, true>(p, out_bf16, num_cus, s);
}

}  // namespace dspark
