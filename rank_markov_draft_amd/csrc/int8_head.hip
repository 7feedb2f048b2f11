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

// Four integers of a row whose scale lies well inside the normal range.  The
// quotient is x times the rounded reciprocal, corrected by its residue (exact
// in a fused product) twice: once to within its last bit, then to the
// division's own rounding; one small enough for its residue to underflow
// rounds to zero anyway, and none is above 127 (1 + 2^-23), by the scale's own
// rounding.  Adding 1.5 * 2^23 rounds to an integer, ties to even, in the
// sum's low bits.  Half a division's instructions: the head's bf16 rows were
// bound by them.
__device__ __forceinline__ bool plain_scale(float s) { return s > 0x1p-100f && s < 0x1p100f; }
__device__ __forceinline__ uint32_t quantize4(float x0, float x1, float x2, float x3, float s, float inv) {
  const float x[4] = {x0, x1, x2, x3};
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float q = x[e] * inv;
    q = __builtin_fmaf(__builtin_fmaf(-q, s, x[e]), inv, q);
    q = __builtin_fmaf(__builtin_fmaf(-q, s, x[e]), inv, q);
    u[e] = __float_as_uint(q + 0x1.8p23f);
  }
  // the low bytes, u[0]'s first
  return __builtin_amdgcn_perm(u[1], u[0], 0x0C0C0400u) | __builtin_amdgcn_perm(u[3], u[2], 0x04000C0Cu);
}

}  // namespace

// LANES threads a row (64 or 256), NV vectors of 8 elements a thread held in
// registers: x is read once.  Bound by HBM: a bf16 head of 129280 rows of 5120
// takes 311 us (6.4 TB/s), an fp32 one 553 us (6.0 TB/s); with a division for
// each element the bf16 one took 391 us.
template <bool BF, int LANES, int NV>
__global__ __launch_bounds__(kQuantThreads) void quantize_rows_kernel(QuantizeParams p) {
  constexpr int NW = BF ? 1 : 2;  // 16-byte words of a vector
  __shared__ uint32_t lds_top[kQuantThreads / 64];
  const int tid = threadIdx.x;
  const int64_t row = (int64_t)blockIdx.x * (kQuantThreads / LANES) + tid / LANES;
  const int t = tid % LANES;
  const bool live = row < p.rows;
  const int d8 = (int)(p.d / 8), q8 = (int)(p.ldq / 8);
  const u32x4_t* const src = (const u32x4_t*)((const char*)p.x + (live ? row : 0) * p.d * (BF ? 2 : 4));
  u32x4_t raw[NV][NW];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = t + j * LANES;
#pragma unroll
    for (int h = 0; h < NW; ++h)
      raw[j][h] = live && i < d8 ? __builtin_nontemporal_load(src + NW * i + h) : u32x4_t{0u, 0u, 0u, 0u};
  }
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int h = 0; h < NW; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = raw[j][h][e];
        // two bf16 values: the magnitudes of the upper half and of the lower
        if constexpr (BF) top = max(top, max(w & 0x7FFF0000u, (w << 16) & 0x7FFF0000u));
        else top = max(top, w & 0x7FFFFFFFu);
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
  const bool plain = plain_scale(s), ok = usable(s);
  const float inv = 1.0f / s;
  uint64_t* const dst = (uint64_t*)(p.q + row * p.ldq);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = t + j * LANES;
    if (i >= q8) break;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (BF) x[e] = (e & 1) ? bf16_hi(raw[j][0][e >> 1]) : bf16_lo(raw[j][0][e >> 1]);
      else x[e] = __uint_as_float(raw[j][e >> 2][e & 3]);
    }
    uint32_t o[2] = {0, 0};
    if (plain) {
#pragma unroll
      for (int h = 0; h < 2; ++h) o[h] = quantize4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3], s, inv);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e >> 2] |= quantize1(x[e], s, ok) << (8 * (e & 3));
    }
    __builtin_nontemporal_store(((uint64_t)o[1] << 32) | o[0], dst + i);  // zeros past d8: the padding
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
// `launch(part)` for parts of at most kLaunchGroups workgroups of `per` rows.
template <bool BF, typename F>
hipError_t by_launches(const QuantizeParams& p, int per, F launch) {
  for (int64_t r0 = 0; r0 < p.rows; r0 += per * kLaunchGroups) {
    QuantizeParams part = p;
    part.x = (const char*)p.x + r0 * p.d * (BF ? 2 : 4);
    part.q = p.q + r0 * p.ldq;
    part.scale = p.scale + r0;
    part.rows = p.rows - r0 < per * kLaunchGroups ? p.rows - r0 : per * kLaunchGroups;
    launch(part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <bool BF, int LANES, int NV>
hipError_t quantize_go(const QuantizeParams& p, hipStream_t s) {
  constexpr int per = kQuantThreads / LANES;
  return by_launches<BF>(p, per, [&](const QuantizeParams& part) {
    hipLaunchKernelGGL((quantize_rows_kernel<BF, LANES, NV>), dim3((unsigned)((part.rows + per - 1) / per)),
                       dim3(kQuantThreads), 0, s, part);
  });
}
template <bool BF>
hipError_t quantize_pick(const QuantizeParams& p, hipStream_t s) {
  // The narrowest form that holds a row: 400000 rows of 512 in bf16 take 109,
  // 155, 260 and 324 us by the four forms in turn, of 2048 387, 465 and 513 us
  // by the last three; 200000 rows of 4096 375 and 397 us.
  // Read twice, 129280 rows of 5120 take 1297 us.
  const bool vec = p.d % 8 == 0 && p.ldq % 8 == 0 && (uintptr_t)p.x % 16 == 0 && (uintptr_t)p.q % 8 == 0;
  if (vec && p.ldq <= 512) return quantize_go<BF, 64, 1>(p, s);
  if (vec && p.ldq <= 2048) return quantize_go<BF, 64, 4>(p, s);
  if (vec && p.ldq <= 4096) return quantize_go<BF, 256, 2>(p, s);
  if (vec && p.ldq <= 8192) return quantize_go<BF, 256, 4>(p, s);
  return by_launches<BF>(p, 1, [&](const QuantizeParams& part) {
    hipLaunchKernelGGL(quantize_rows_any_kernel<BF>, dim3((unsigned)part.rows), dim3(kQuantThreads), 0, s, part);
  });
}
}  // namespace

hipError_t launch_quantize_rows(const QuantizeParams& p, bool bf16, hipStream_t s) {
  if (p.rows > 0x7FFFFFFF) return hipErrorNotSupported;
  return bf16 ? quantize_pick<true>(p, s) : quantize_pick<false>(p, s);
}

// ---------------------------------------------------------------- product
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));  // rows of the output start at any element

// A workgroup of WM x WN waves owns tiles of 32 MI WM rows x 32 NJ WN
// vocabulary columns and walks them in a persistent loop; a wave holds MI x
// NJ blocks of 32 x 32 sums.  The inner dimension is cut into chunks of 128
// bytes; a chunk's rows of q and of the head are loaded straight into LDS
// (16 bytes a lane, no registers), up to STAGES chunks at a time.  A row's
// eight 16-byte pieces sit at positions piece ^ (row % 8), so that the
// fragment reads of eight consecutive rows fall on different banks (even so
// the counters call 0.48 of LDS's access cycles conflicts).  The chunk stream
// runs on across tiles.
//
// v_mfma_i32_32x32x32_i8: rows of q on M, vocabulary columns on N.
//
// AHEAD (tiles bound by the matrix cores): the fragments of a product are
// read while the product before it runs, and the hand-over from chunk to
// chunk (wait, barrier, first reads) runs behind the chunk's last products.
// Otherwise (tiles bound by the head's stream) all of a chunk's fragments are
// read at once, so that their latency is paid once a chunk.
//
// PIECE: the head goes straight to LDS 16 bytes a lane where its rows are
// whole 16-byte pieces, else 4 bytes a lane where they are whole words, else
// through registers by unaligned loads, a chunk ahead (0).  Whole calls, in us,
// by pieces of 16 bytes, words and registers: 37 rows at V = 32003, d = 2056
// (2048 for the first) 19, 20, 26; at V = 129280, d = 5124 (5120) 1 row 114,
// 148, 159; 128 rows 141, 181, 211; 320 rows 228, 278, 388.
template <int MI, int NJ, int WM, int WN, int STAGES, bool AHEAD, int PIECE, bool OBF>
__global__ __launch_bounds__(64 * WM * WN) void int8_head_kernel(Int8HeadParams p, int row_tiles, int tiles) {
  constexpr int NW = WM * WN, THREADS = 64 * NW;
  constexpr int BM = 32 * MI * WM, BN = 32 * NJ * WN, BK = (int)kInt8K;
  constexpr int STAGE = (BM + BN) * BK;
  constexpr bool DIRECT = PIECE != 0;
  // load instructions of a chunk per wave, of 8 rows each (2 of the head's by words)
  constexpr int RB = PIECE == 4 ? 2 : 8, PA = BM / 8 / NW, PB = DIRECT ? BN / RB / NW : 0, PER = PA + PB;
  constexpr int REGS = DIRECT ? 1 : BN * 8 / THREADS;    // pieces of the head a thread moves itself
  static_assert(BM / 8 % NW == 0 && BN / 8 % NW == 0, "whole load instructions per wave");
  static_assert(PIECE != 4 || RB * NW % 8 == 0, "a lane's swizzle is the same for all its rows");
  static_assert(DIRECT || (STAGES == 2 && !AHEAD), "register pieces are one chunk ahead");
  static_assert((STAGES - 1) * PER < 64, "wait count");
  // a wave's part of the output on its way to memory: ER rows x 32 NJ columns
  constexpr int OS = OBF ? 2 : 4, ER = OBF ? 16 : 8, EROW = 32 * NJ * OS, EBYTES = ER * EROW;
  __shared__ __attribute__((aligned(16))) unsigned char lds[STAGES * STAGE + NW * EBYTES];

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

  // ---- the load stream
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
  // load instruction j of this wave fills rows 8 (wave + j NW) .. + 7, lane l
  // the position l % 8 of row l / 8 (which holds piece l % 8 ^ row % 8)
  const uint32_t row8 = 8u * (uint32_t)wave + (uint32_t)(lane >> 3);
  const uint32_t q16 = 16u * (uint32_t)((lane & 7) ^ (lane >> 3));
  const uint32_t offa = row8 * (uint32_t)p.ldx + q16;
  // by words: rows 2 (wave + j NW) and the next, lane l word l % 32 of a row
  const uint32_t row2 = 2u * (uint32_t)wave + (uint32_t)(lane >> 5);
  const uint32_t offb = PIECE == 4 ? row2 * (uint32_t)p.d + 16u * ((uint32_t)(lane >> 2 & 7) ^ (row2 & 7)) + 4u * (uint32_t)(lane & 3)
                                   : row8 * (uint32_t)p.d + q16;
  u32x4_t held[REGS];
  auto issue = [&](int g) __attribute__((always_inline)) {  // chunk g of the stream, in order
    const bool live = g < total;
    const uint32_t k0 = (uint32_t)lc * BK;
    const uint32_t stage = lds_address(&lds[(uint32_t)(g % STAGES) * STAGE]);
#pragma unroll
    for (int j = 0; j < PA; ++j)
      load_lds16(ba, live ? offa + (uint32_t)(8 * NW * j) * (uint32_t)p.ldx + k0 : kBufferOob,
                 stage + 1024u * (uint32_t)(wave + NW * j));
#pragma unroll
    for (int j = 0; j < PB; ++j) {
      const uint32_t off = live ? offb + (uint32_t)(RB * NW * j) * (uint32_t)p.d + k0 : kBufferOob;
      const uint32_t to = stage + BM * BK + (uint32_t)(RB * BK) * (uint32_t)(wave + NW * j);
      if constexpr (PIECE == 4) load_lds4(bb, off, to);
      else load_lds16(bb, off, to);
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

  // ---- the products: fragments of the wave's MI x NJ blocks for one matrix
  // instruction each
  constexpr int S = BK / 32;
  struct Frags {
    i32x4_t a[MI], b[NJ];
  };
  auto read = [&](int g, int s, Frags& f) __attribute__((always_inline)) {  // step s of chunk g
    const unsigned char* const st = &lds[(g % STAGES) * STAGE + 16 * ((2 * s + (lane >> 5)) ^ (lane & 7))];
#pragma unroll
    for (int i = 0; i < MI; ++i) f.a[i] = *(const i32x4_t*)(st + (32 * (MI * wm + i) + (lane & 31)) * BK);
#pragma unroll
    for (int j = 0; j < NJ; ++j) f.b[j] = *(const i32x4_t*)(st + (BM + 32 * (NJ * wn + j) + (lane & 31)) * BK);
  };
  i32x16_t acc[MI][NJ];
  auto multiply = [&](const Frags& f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
  };

  if (my == 0) return;
  bind(0);
  issue(0);
  put(0);
#pragma unroll
  for (int g = 1; g < STAGES - (AHEAD ? 0 : 1); ++g) issue(g);
  Frags f[AHEAD ? 2 : S];
  if constexpr (AHEAD) {
    wait_vmcnt<(STAGES - 1) * PER>();
    lds_barrier();
    read(0, 0, f[0]);
  }
  int g = 0, landed = 0;  // landed: steps whose chunk is known to have arrived
  for (int t = 0; t < my; ++t) {
    const int tile = first + t * G;
    const int64_t r0 = (int64_t)(tile % row_tiles) * BM + 32 * MI * wm;
    const int64_t v0 = (int64_t)(tile / row_tiles) * BN + 32 * NJ * wn;
    // The scales of the lane's columns are loaded here, and those of its rows
    // (the same for half a wave) by scalar loads at the end: a vector load
    // that some path leaves unused would make the compiler wait for all
    // memory inside the chunk loop.
    float wsc[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int64_t v = v0 + 32 * j + (lane & 31);
      wsc[j] = p.ws[v < p.V ? v : p.V - 1];
    }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
    for (int c = 0; c < C; ++c, ++g) {
      if constexpr (AHEAD) {
#pragma unroll
        for (int s = 0; s < S - 1; ++s) {
          read(g, s + 1, f[(s + 1) & 1]);
          multiply(f[s & 1]);
        }
        // The chunk's last products run behind the hand-over to the next: its
        // loads have landed for every wave, every wave has read all of this
        // chunk, whose stage takes the loads of chunk g + STAGES.
        wait_vmcnt<(STAGES - 2) * PER>();
        lds_barrier();
        read(g + 1, 0, f[0]);  // before the loads, which would hold up LDS
        issue(g + STAGES);
        multiply(f[(S - 1) & 1]);
      } else {
        // chunk g has landed for every wave, and every wave has read chunk g - 1
        if (landed > 0) --landed;
        else wait_vmcnt<(STAGES - 2) * PER>();
        lds_barrier();
        issue(g + STAGES - 1);
#pragma unroll
        for (int s = 0; s < S; ++s) read(g, s, f[s]);
#pragma unroll
        for (int s = 0; s < S; ++s) multiply(f[s]);
        put(g + 1);
      }
    }
    if constexpr (!AHEAD) {
      // the chunks on their way (the last was issued a step ago), so that the
      // next steps need not wait for the stores
      wait_vmcnt<0>();
      landed = STAGES - 1;
    }
    // The tile's sums times its scales.  Lane l holds column l % 32 of rows
    // 8 (e / 4) + 4 (l / 32) + e % 4 of each block, which as they are would
    // leave in stores of one element a lane (a ninth of the whole time at
    // 2560 rows).  So ER rows at a time go through the wave's own LDS, in
    // 16-byte pieces, those of every other four rows moved by half a row so
    // that both halves of the wave write to different banks, and leave in
    // whole pieces of consecutive columns.
    unsigned char* const mine = &lds[STAGES * STAGE + wave * EBYTES];
    constexpr int PIECES = EROW / 16, HALF = PIECES / 2;  // of a row
    constexpr int SETS = ER / 8;                          // groups of 8 rows in an exchange
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int x = 0; x < 4 / SETS; ++x) {
        const int64_t rb = r0 + 32 * i + ER * x;  // first row of the exchange
        if (rb >= p.rows) continue;
#pragma unroll
        for (int u = 0; u < SETS; ++u) {
          const int lr = 8 * u + 4 * (lane >> 5);  // first of the lane's four rows
          const auto* const xs = (const __attribute__((address_space(4))) float*)(p.xs + rb + 8 * u);
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              const float y = ((lane >> 5 ? xs[4 + e] : xs[e]) * wsc[j]) * (float)acc[i][j][4 * (SETS * x + u) + e];
              const int byte = (32 * j + (lane & 31)) * OS;
              unsigned char* const at = mine + (lr + e) * EROW + 16 * ((byte >> 4) ^ (HALF * (lane >> 5))) + (byte & 15);
              if constexpr (OBF) *(uint16_t*)at = (uint16_t)(pack_bf16x2(y, 0.0f) & 0xFFFFu);
              else *(float*)at = y;
            }
        }
#pragma unroll
        for (int h = 0; h < ER * PIECES / 64; ++h) {
          const int pc = lane + 64 * h, lr = pc / PIECES, q = pc % PIECES;
          const u32x4_t w = *(const u32x4_t*)(mine + lr * EROW + 16 * (q ^ (HALF * (lr >> 2 & 1))));
          const int64_t n = rb + lr, v = v0 + q * (16 / OS);
          if (n < p.rows && v < p.V) {
            unsigned char* const dst = (unsigned char*)p.out + (n * p.V + v) * OS;
            if (v + 16 / OS <= p.V) {
              __builtin_nontemporal_store(w, (u32x4_any_t*)dst);
            } else {
              for (int e = 0; e < (int)(p.V - v); ++e) {
                if constexpr (OBF) ((uint16_t*)dst)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                else ((uint32_t*)dst)[e] = w[e];
              }
            }
          }
        }
      }
  }
  wait_vmcnt<0>();
}

namespace {
template <int MI, int NJ, int WM, int WN, int STAGES, bool AHEAD, int PIECE>
hipError_t head_go(const Int8HeadParams& p, bool obf, int groups, hipStream_t s) {
  constexpr int BM = 32 * MI * WM, BN = 32 * NJ * WN;
  const int64_t rt = (p.rows + BM - 1) / BM, tiles = rt * ((p.V + BN - 1) / BN);
  if (tiles > 0x3FFFFFFF || rt > 0x3FFFFFFF) return hipErrorNotSupported;
  // persistent: a workgroup's chunk count is an int
  if ((tiles / groups + 1) * (p.ldx / kInt8K) > 0x3FFFFFFF) return hipErrorNotSupported;
  const dim3 grid((unsigned)(tiles < groups ? tiles : groups)), block(64 * WM * WN);
  if (obf)
    hipLaunchKernelGGL((int8_head_kernel<MI, NJ, WM, WN, STAGES, AHEAD, PIECE, true>), grid, block, 0, s, p, (int)rt,
                       (int)tiles);
  else
    hipLaunchKernelGGL((int8_head_kernel<MI, NJ, WM, WN, STAGES, AHEAD, PIECE, false>), grid, block, 0, s, p, (int)rt,
                       (int)tiles);
  return hipGetLastError();
}
}  // namespace

// The forms of the kernel, and what a round of their tiles over the CUs takes
// beside one another (us at d = 5120, the one hidden size at which they were
// timed against each other; tiles sharing the head's rows; a round
// of one tile a CU, or of two where two workgroups fit).  Small tiles win
// where a larger one would compute rows that do not exist or leave CUs
// without a tile, large ones by their rate: the form with the shortest sum
// of rounds is taken.  At V = 129280, in us (128x256, 192x256, 256x256,
// 320x256 tiles): 128 rows 132, 155, 167, 188; 192 rows 192, 163, 180, 195;
// 256 rows 204, 259, 186, 204; 320 rows 268, 269, 311, 211.  64 rows:
// 121 with 64x256 tiles, 171 with 32x128; one row at V = 32003 as well as
// 37 rows are fastest with the smallest tiles that cover them.
namespace {
struct Form {
  int bm, bn, per_cu;
  float round;
};
constexpr Form kDirect[] = {{32, 128, 1, 14.0f},  {64, 128, 1, 19.0f},  {64, 256, 1, 32.0f}, {128, 256, 1, 45.0f},
                            {192, 256, 1, 59.0f}, {256, 256, 1, 78.0f}, {320, 256, 1, 90.0f}};
constexpr Form kStaged[] = {{64, 128, 2, 48.0f}, {128, 256, 1, 68.0f}, {192, 256, 1, 78.0f}, {256, 256, 1, 92.0f}};

template <int N>
int pick_form(const Form (&forms)[N], int64_t rows, int64_t V, int num_cus) {
  int best = 0;
  double least = 0.0;
  for (int i = 0; i < N; ++i) {
    const Form& f = forms[i];
    const int64_t tiles = ((rows + f.bm - 1) / f.bm) * ((V + f.bn - 1) / f.bn), slots = (int64_t)num_cus * f.per_cu;
    const double cost = (double)((tiles + slots - 1) / slots) * f.round;
    if (i == 0 || cost < least) {
      best = i;
      least = cost;
    }
  }
  return best;
}
}  // namespace

namespace {
template <int PIECE>
hipError_t head_direct(const Int8HeadParams& p, bool out_bf16, int num_cus, hipStream_t s) {
  switch (pick_form(kDirect, p.rows, p.V, num_cus)) {
    case 0: return head_go<1, 1, 1, 4, 4, false, PIECE>(p, out_bf16, num_cus, s);
    case 1: return head_go<1, 1, 2, 4, 4, false, PIECE>(p, out_bf16, num_cus, s);
    case 2: return head_go<1, 2, 2, 4, 3, false, PIECE>(p, out_bf16, num_cus, s);
    case 3: return head_go<2, 2, 2, 4, 3, true, PIECE>(p, out_bf16, num_cus, s);
    case 4: return head_go<3, 2, 2, 4, 2, true, PIECE>(p, out_bf16, num_cus, s);
    case 5: return head_go<4, 2, 2, 4, 2, true, PIECE>(p, out_bf16, num_cus, s);
    default: return head_go<5, 2, 2, 4, 2, true, PIECE>(p, out_bf16, num_cus, s);
  }
}
}  // namespace

hipError_t launch_int8_head(const Int8HeadParams& p, bool out_bf16, int num_cus, hipStream_t s) {
  if (num_cus < 1 || p.d > kInt8MaxInner || p.ldx % kInt8K != 0 || p.ldx < p.d) return hipErrorNotSupported;
  if (p.d % 16 == 0 && (uintptr_t)p.wq % 16 == 0) return head_direct<16>(p, out_bf16, num_cus, s);
  if (p.d % 4 == 0 && (uintptr_t)p.wq % 4 == 0) return head_direct<4>(p, out_bf16, num_cus, s);
  switch (pick_form(kStaged, p.rows, p.V, num_cus)) {
    case 0: return head_go<1, 1, 2, 4, 2, false, 0>(p, out_bf16, 2 * num_cus, s);
    case 1: return head_go<2, 2, 2, 4, 2, false, 0>(p, out_bf16, num_cus, s);
    case 2: return head_go<3, 2, 2, 4, 2, false, 0>(p, out_bf16, num_cus, s);
    default: return head_go<4, 2, 2, 4, 2, false, 0>(p, out_bf16, num_cus, s);
  }
}

}  // namespace dspark
