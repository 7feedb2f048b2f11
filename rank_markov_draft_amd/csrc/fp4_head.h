// fp4_head.h -- interface of the 4-bit vocabulary head (fp4_head.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dspark {

// Blocks of 32 numbers as 4-bit codes (e2m1, two a byte, the first in the low
// half) with one biased power of two (e8m0) a block.  A row of d numbers holds
// fp4_blocks(d) blocks, past d filled up with zeros.
inline int64_t fp4_blocks(int64_t d) { return (d / 128 + (d % 128 != 0)) * 4; }

struct Fp4QuantizeParams {
  const void* x;       // [rows, d]
  uint8_t* codes;      // [rows, ldc] bytes, 16-byte aligned, ldc a multiple of 64
  uint8_t* scales;     // [rows, lds] bytes, 4-byte aligned, lds = ldc / 16
  int64_t rows;
  int64_t d;
  int64_t ldc;
};
hipError_t launch_fp4_quantize(const Fp4QuantizeParams& p, bool bf16, hipStream_t s);

struct Fp4DequantizeParams {
  const uint8_t* codes;   // [rows, 16 * blocks]
  const uint8_t* scales;  // [rows, blocks]
  void* x;                // [rows, d]
  int64_t rows;
  int64_t d;
  int64_t blocks;
};
hipError_t launch_fp4_dequantize(const Fp4DequantizeParams& p, bool bf16, hipStream_t s);

// out[n, v] = sum_b 2^(xs[n, b] + ws[v, b] - 254) sum_i xc[n, 32 b + i] wc[v, 32 b + i].
constexpr int64_t kFp4K = 128;               // code bytes of a chunk (256 numbers, 8 blocks)
constexpr int64_t kFp4MaxInner = 1 << 20;    // a tile's rows stay within one buffer
struct Fp4HeadParams {
  const uint8_t* xc;  // [rows, ldx], 16-byte aligned; ldx a multiple of kFp4K, zeros past the row's blocks
  const uint8_t* xs;  // [rows, ldx / 16], 4-byte aligned
  const uint8_t* wc;  // [V, 16 * blocks], 16-byte aligned
  const uint8_t* ws;  // [V, blocks], 4-byte aligned
  void* out;          // [rows, V] fp32 or bf16
  int64_t rows;
  int64_t V;
  int64_t blocks;     // a multiple of 4
  int64_t ldx;
};
hipError_t launch_fp4_head(const Fp4HeadParams& p, bool out_bf16, int num_cus, hipStream_t s);

}  // namespace dspark
