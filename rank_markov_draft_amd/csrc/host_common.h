// host_common.h -- host-side pieces shared by the translation units of the C
// ABI (dspark_markov.hip, dspark_serving.hip): the workspace layout, size
// arithmetic and argument checks.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <string>

#include "dspark_markov.h"
#include "markov_kernels.h"

namespace dspark {

// Message of this thread's last failure (dspark_markov_last_error); defined
// in dspark_markov.hip.
void set_last_error(const std::string& msg);

namespace host {

// Workspace layout (the same for every call, so calls of different shapes
// may share a workspace):
//   [0, 256)      control block: the device error word, the
//                 synchronisation-failure count of the persistent chain and
//                 its test hook, each on its own 64-byte line;
//   chain area    arrival counters (kChainSyncBytes), then the device-wide
//                 argmax keys per (step, key group, row): 64-byte slots for
//                 up to kChainMaxSteps steps of 64 rows (greedy chain), or
//                 16-byte slots for up to 4096 step-rows (temperature
//                 chain).  Only the persistent chains write here, and they
//                 leave the area zeroed: their keys and counters must start
//                 at zero, so no other path may put data in it;
//   data          from kDataOffset: the apply kernels' store sink, or the
//                 sampling steps' per-(row, vocabulary slice) argmax keys
//                 (B * ceil(V/128) words), or the backward's and the gated
//                 head's scratch.
constexpr size_t kControlBytes = 256;
constexpr int64_t kChainMaxSteps = 16;
constexpr size_t kChainAreaBytes =
    dspark::kChainSyncBytes + (size_t)kChainMaxSteps * 8 * 64 * dspark::kKeyPad * sizeof(uint64_t);
constexpr size_t kDataOffset = kControlBytes + kChainAreaBytes;
static_assert(kDataOffset % 256 == 0, "data region alignment");

struct Control {
  uint32_t bad_rows;       // byte 0: rows with out-of-range ids
  uint32_t pad0[15];
  uint32_t sync_failures;  // byte 64: failed device-wide waits of the persistent chain
  uint32_t pad1[15];
  uint32_t chain_test_hook;  // byte 128: nonzero makes the chain's waits give up at once
  uint32_t pad2[15];
};
static_assert(sizeof(Control) <= kControlBytes, "control block");

// Size arithmetic of the workspace queries saturates at SIZE_MAX, the
// answer for sizes that cannot be represented.
inline size_t add_sz(size_t a, size_t b) {
  size_t o;
  return __builtin_add_overflow(a, b, &o) ? SIZE_MAX : o;
}
inline size_t mul_sz(size_t a, size_t b) {
  size_t o;
  return __builtin_mul_overflow(a, b, &o) ? SIZE_MAX : o;
}
inline size_t align256(size_t x) { return x > SIZE_MAX - 255 ? SIZE_MAX : (x + 255) & ~(size_t)255; }

inline size_t partials_bytes(int64_t B, int64_t V) {
  return align256(mul_sz(mul_sz((size_t)B, (size_t)(V / 128 + (V % 128 != 0))), sizeof(uint64_t)));
}

// Compute units of the current device, cached per device.
inline int device_cus() {
  static int cache[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
  if (cache[dev] == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return 0;
    cache[dev] = prop.multiProcessorCount;
  }
  return cache[dev];
}

inline dspark_status_t device_failure(hipError_t e, const char* what) {
  set_last_error(std::string(what) + ": " + hipGetErrorString(e));
  return DSPARK_ERR_DEVICE;
}

inline bool known_dtype(int d) { return d == DSPARK_F32 || d == DSPARK_BF16; }

inline size_t dtype_bytes(dspark_dtype_t d) { return d == DSPARK_F32 ? 4 : 2; }

inline bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Byte ranges [a, a+na) and [b, b+nb) intersect.
inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

inline int64_t vocab_slices(int64_t V) { return (V + 127) / 128; }

// Largest rank the row-tile kernels take (they walk the rank in chunks; the
// limit is the documented one of the C ABI).
constexpr int64_t kGenericMaxRank = 16384;

// The bf16 tile kernel takes the call when both dtypes are bf16, the rank is
// a multiple of 8 no larger than 512, rows of logits are whole 16-byte
// vectors and every streamed pointer is 16-byte aligned.
inline bool tile_path(dspark_dtype_t ldt, dspark_dtype_t wdt, int64_t V, int64_t r, const void* base,
               const void* out, const void* w1, const void* w2) {
  return ldt == DSPARK_BF16 && wdt == DSPARK_BF16 && r % 8 == 0 &&
         dspark::tile_ks_for_rank(r) != 0 && V % 8 == 0 && aligned16(base) &&
         (out == nullptr || aligned16(out)) && aligned16(w1) && aligned16(w2);
}

// Shared checks of both operations.  Returns DSPARK_OK to proceed, or the
// status to return; *empty is set when there is no work.
inline dspark_status_t check_common(int ldt, int wdt, int64_t B, int64_t M, int64_t V, int64_t r,
                             int64_t* elems) {
  if (!known_dtype(ldt) || !known_dtype(wdt)) return DSPARK_ERR_INVALID_ARGUMENT;
  if (B < 0 || M < 0 || V < 0 || r <= 0) return DSPARK_ERR_INVALID_ARGUMENT;
  int64_t rows = 0, e = 0, wv = 0;
  if (!mul_ok(B, M, &rows) || !mul_ok(rows, V, &e) || !mul_ok(V, r, &wv))
    return DSPARK_ERR_INVALID_ARGUMENT;
  if (V > (int64_t)0x7FFFFFFF) return DSPARK_ERR_UNSUPPORTED;
  *elems = e;
  return DSPARK_OK;
}

}  // namespace host
}  // namespace dspark
