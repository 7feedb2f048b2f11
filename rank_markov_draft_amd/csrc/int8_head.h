// int8_head.h -- interface of the 8-bit vocabulary head (int8_head.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dspark {

// Rows of x [rows, d] as 8-bit integers with one scale each.  Row n of q
// starts at q + n * ldq (ldq >= d); the bytes d .. ldq - 1 are zeroed.
struct QuantizeParams {
  const void* x;
  int8_t* q;
  float* scale;  // [rows]
  int64_t rows;
  int64_t d;
  int64_t ldq;
};
hipError_t launch_quantize_rows(const QuantizeParams& p, bool bf16, hipStream_t s);

// out[n, v] = (xs[n] * ws[v]) * sum_i xq[n, i] wq[v, i].
constexpr int64_t kInt8K = 128;          // inner bytes of a chunk: ldx is a multiple
constexpr int64_t kInt8RowPad = 512;     // readable floats past xs[rows - 1]
constexpr int64_t kInt8MaxInner = 131072;  // 127 * 127 * d stays below 2^31
struct Int8HeadParams {
  const int8_t* xq;  // [rows, ldx], 16-byte aligned, zeros past d
  const float* xs;   // [rows], 16-byte aligned, kInt8RowPad more floats readable
  const int8_t* wq;  // [V, d]
  const float* ws;   // [V]
  void* out;         // [rows, V] fp32 or bf16
  int64_t rows;
  int64_t V;
  int64_t d;
  int64_t ldx;
};
hipError_t launch_int8_head(const Int8HeadParams& p, bool out_bf16, int num_cus, hipStream_t s);

}  // namespace dspark
