// distill.hip -- distillation of the drafter's logits from a teacher's top
// logits (gfx950).
//
// For a row of logits x over the vocabulary and the teacher's list of ids i_j
// with logits t_j (entries with an id outside [0, V) or a logit of -inf do not
// count), at temperature tau,
//     q = softmax(t / tau) over the list,   p = softmax(x / tau) over the vocabulary,
//     loss   = tau^2 sum_j q_j (log q_j - log p[i_j]),
//     dloss / dx[v] = tau (p[v] - sum_{j: i_j = v} q_j).
// Both passes stream the row once: the forward one with a running maximum and
// sum, the backward one from the statistics that the forward one left.
#include "device_common.h"
#include "distill.h"

namespace dspark {

namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;                      // columns a lane takes at once
constexpr int kGroup = kThreads * kVec;      // columns a workgroup takes at once
constexpr int kAhead = 4;                    // vectors a lane loads before it uses the first
constexpr int kBackSlice = kGroup * kAhead;  // columns of a backward workgroup
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));  // rows start at any element

// Eight columns of a row from column v on, as loaded; -inf past its end.
template <bool BF>
struct Vec {
  u32x4_t w[BF ? 1 : 2];
};
template <bool BF>
__device__ __forceinline__ Vec<BF> load_vec(const void* row, int64_t v, int64_t V) {
  Vec<BF> r;
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
__device__ __forceinline__ float at(const Vec<BF>& r, int e) {
  if constexpr (BF) return (e & 1) ? bf16_hi(r.w[0][e >> 1]) : bf16_lo(r.w[0][e >> 1]);
  else return __uint_as_float(r.w[e >> 2][e & 3]);
}
template <bool BF>
__device__ __forceinline__ float load_one(const void* row, int64_t v) {
  return BF ? bf16_lo(((const uint16_t*)row)[v]) : ((const float*)row)[v];
}

// Weight 2^((x - m) kappa) of a logit: the difference first, so that the
// largest ones, which make up the sum, are the most exact.  m is a number
// (the type's lowest where a row has none), so -inf weighs nothing.
__device__ __forceinline__ float weight(float x, float m, float kappa) {
  return __builtin_amdgcn_exp2f((x - m) * kappa);
}
constexpr float kLowest = -3.40282347e38f;

// The largest logit and the sum of weights relative to it of a set of columns.
struct Sum {
  float m, z;
};
__device__ __forceinline__ Sum join(Sum a, Sum b, float kappa) {
  const float m = fmaxf(a.m, b.m);
  return Sum{m, a.z * weight(a.m, m, kappa) + b.z * weight(b.m, m, kappa)};
}
__device__ __forceinline__ Sum wave_join(Sum s, float kappa) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1)
    s = join(s, Sum{__shfl_xor(s.m, off, 64), __shfl_xor(s.z, off, 64)}, kappa);
  return s;
}
__device__ __forceinline__ double wave_sum_f64(double x) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
  return x;
}

// The sum of a workgroup's columns [v0, v1), valid in every thread.
template <bool BF>
__device__ __forceinline__ Sum slice_sum(const void* row, int64_t v0, int64_t v1, int64_t V, float kappa, Sum* lds) {
  Sum s{kLowest, 0.0f};
  for (int64_t v = v0 + threadIdx.x * kVec; v < v1; v += kAhead * kGroup) {
    Vec<BF> r[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) r[j] = load_vec<BF>(row, v + j * kGroup < v1 ? v + j * kGroup : V, V);
    float m = s.m;
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int e = 0; e < kVec; ++e) m = fmaxf(m, at<BF>(r[j], e));
    float z = 0.0f;  // of these 32 columns first: 32 times fewer roundings of the long sum
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int e = 0; e < kVec; ++e) z += weight(at<BF>(r[j], e), m, kappa);
    s.z = s.z * weight(s.m, m, kappa) + z;
    s.m = m;
  }
  s = wave_join(s, kappa);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  s = lds[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) s = join(s, lds[w], kappa);
  return s;
}

// Loss and statistics of a row whose sum is known, by a whole workgroup, in 64
// bits: it is a small difference of large terms.
template <bool BF>
__device__ __forceinline__ void finish_row(const DistillParams& p, int64_t n, float m, double z, double* lds) {
  const char* const row = (const char*)p.logits + n * p.V * (BF ? 2 : 4);
  const int64_t* const ids = p.teacher_ids + n * p.K;
  auto teacher = [&](int j) __attribute__((always_inline)) {
    return p.teacher_bf16 ? bf16_lo(((const uint16_t*)p.teacher_logits)[n * p.K + j])
                          : ((const float*)p.teacher_logits)[n * p.K + j];
  };
  auto counts = [&](int j, float t) __attribute__((always_inline)) {
    const int64_t id = ids[j];
    return id >= 0 && id < p.V && t != -__builtin_inff();
  };
  const int K = (int)p.K, tid = threadIdx.x;
  float top = kLowest;
  bool any = false;
  for (int j = tid; j < K; j += kThreads) {
    const float t = teacher(j);
    if (counts(j, t)) {
      any = true;
      top = fmaxf(top, t);
    }
  }
  top = __shfl(wave_max_f32_to_lane63(top), 63, 64);
  __shared__ float lds_top[kThreads / 64];
  __shared__ int lds_any;
  if (tid == 0) lds_any = 0;
  __syncthreads();
  if ((tid & 63) == 0) lds_top[tid >> 6] = top;
  if (any) lds_any = 1;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) top = fmaxf(top, lds_top[w]);
  // with u = t / tau - top / tau and y = x / tau - m / tau: q = e^u / zt and
  // the loss is sum_j q_j (u_j - y_j) - log zt + log z, times tau^2
  double zt = 0.0, cross = 0.0;
  for (int j = tid; j < K; j += kThreads) {
    const float t = teacher(j);
    if (!counts(j, t)) continue;
    const double u = ((double)t - (double)top) / p.tau, e = exp(u);
    zt += e;
    if (e != 0.0) cross += e * (u - ((double)load_one<BF>(row, ids[j]) - (double)m) / p.tau);
  }
  zt = wave_sum_f64(zt);
  cross = wave_sum_f64(cross);
  if ((tid & 63) == 0) {
    lds[2 * (tid >> 6)] = zt;
    lds[2 * (tid >> 6) + 1] = cross;
  }
  __syncthreads();
  if (tid == 0) {
    zt = cross = 0.0;
    for (int w = 0; w < kThreads / 64; ++w) {
      zt += lds[2 * w];
      cross += lds[2 * w + 1];
    }
    double loss = 0.0;
    // a row with nothing above -inf has no distribution: the teacher's lies
    // wholly where it has none
    if (lds_any) loss = z == 0.0 ? __builtin_inf() : p.tau * p.tau * (cross / zt - log(zt) + log(z));
    p.loss[n] = (float)loss;
    float* const st = p.stats + 4 * n;
    st[0] = m;
    st[1] = (float)z;
    st[2] = top;
    st[3] = lds_any ? (float)zt : 0.0f;
  }
}

}  // namespace

// One workgroup a slice of a row; with one slice it finishes the row.  Rows are
// cut only until the device is full (2048 workgroups).  Bound by HBM: 4096 rows
// of 129280 in bf16 take 196 us (5.4 TB/s), 320 rows in six slices each 17 us
// and 4.5 us more for their finish.
template <bool BF>
__global__ __launch_bounds__(kThreads) void distill_sum_kernel(DistillParams p, int64_t r0, int slices, int64_t slice) {
  __shared__ Sum lds[kThreads / 64];
  __shared__ double lds64[2 * (kThreads / 64)];
  const int64_t n = r0 + blockIdx.x / (unsigned)slices;
  const int i = (int)(blockIdx.x % (unsigned)slices);
  const char* const row = (const char*)p.logits + n * p.V * (BF ? 2 : 4);
  const int64_t v0 = i * slice, v1 = v0 + slice < p.V ? v0 + slice : p.V;
  const Sum s = slice_sum<BF>(row, v0, v1, p.V, p.kappa, lds);
  if (slices == 1) {
    finish_row<BF>(p, n, s.m, (double)s.z, lds64);
  } else if (threadIdx.x == 0) {
    float* const out = p.partials + 2 * (n * slices + i);
    out[0] = s.m;
    out[1] = s.z;
  }
}

template <bool BF>
__global__ __launch_bounds__(kThreads) void distill_finish_kernel(DistillParams p, int64_t r0, int slices) {
  __shared__ double lds64[2 * (kThreads / 64)];
  const int64_t n = r0 + blockIdx.x;
  // every wave joins the slices by itself
  const int lane = threadIdx.x & 63;
  float m = kLowest;
  for (int i = lane; i < slices; i += 64) m = fmaxf(m, p.partials[2 * (n * slices + i)]);
  m = __shfl(wave_max_f32_to_lane63(m), 63, 64);
  double z = 0.0;
  for (int i = lane; i < slices; i += 64) {
    const float* const q = p.partials + 2 * (n * slices + i);
    z += (double)q[1] * (double)weight(q[0], m, p.kappa);
  }
  finish_row<BF>(p, n, m, wave_sum_f64(z), lds64);
}

// A workgroup writes kBackSlice columns of a row's gradient: g tau p for all of
// them, then the columns that stand in the teacher's list over again with its
// weight taken off.  Their logits are loaded before anything is written, so
// the gradient may take the logits' place.  Bound by HBM: 4096 rows of 129280 in
// bf16 (2.1 GB) take 377 us (5.6 TB/s), 320 rows 32 us.
template <bool BF>
__global__ __launch_bounds__(kThreads) void distill_backward_kernel(DistillParams p, int64_t r0, unsigned slices) {
  constexpr int PER = (int)(kDistillMaxEntries / kThreads);
  __shared__ int64_t ids[kDistillMaxEntries];
  __shared__ float weights[kDistillMaxEntries];
  const int64_t n = r0 + blockIdx.x / slices;
  const int64_t v0 = (int64_t)(blockIdx.x % slices) * kBackSlice;
  const int64_t v1 = v0 + kBackSlice < p.V ? v0 + kBackSlice : p.V;
  const int tid = threadIdx.x, K = (int)p.K;
  const float* const st = p.stats + 4 * n;
  const float m = st[0], z = st[1], top = st[2], zt = st[3];
  const char* const row = (const char*)p.logits + n * p.V * (BF ? 2 : 4);
  char* const out = (char*)p.grad + n * p.V * (BF ? 2 : 4);
  const bool live = zt != 0.0f && z != 0.0f;  // (NaN is live)
  const float gt = live ? (float)((double)p.grad_loss[n] * p.tau) : 0.0f;
  Vec<BF> r[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int64_t v = v0 + tid * kVec + j * kGroup;
    r[j] = load_vec<BF>(row, v < v1 ? v : p.V, p.V);
  }
  float own[PER];
  if (live) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = tid + i * kThreads;
      own[i] = 0.0f;
      if (j < K) {
        const int64_t id = p.teacher_ids[n * p.K + j];
        const float t = p.teacher_bf16 ? bf16_lo(((const uint16_t*)p.teacher_logits)[n * p.K + j])
                                       : ((const float*)p.teacher_logits)[n * p.K + j];
        const bool counts = id >= v0 && id < v1 && t != -__builtin_inff();
        ids[j] = counts ? id : -1;
        if (counts) {
          weights[j] = (float)(exp(((double)t - (double)top) / p.tau) / (double)zt);
          own[i] = load_one<BF>(row, id);
        }
      }
    }
  }
  const float scale = gt / z;
  wait_vmcnt<0>();  // every logit that the workgroup needs is here
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int64_t v = v0 + tid * kVec + j * kGroup;
    if (v >= v1) continue;
    float y[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) y[e] = live ? weight(at<BF>(r[j], e), m, p.kappa) * scale : 0.0f;
    if (v + kVec <= p.V) {
      u32x4_any_t* const dst = (u32x4_any_t*)(out + v * (BF ? 2 : 4));
      if constexpr (BF) {
        __builtin_nontemporal_store(u32x4_t{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                            pack_bf16x2(y[6], y[7])}, dst);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          __builtin_nontemporal_store(u32x4_t{__float_as_uint(y[4 * h]), __float_as_uint(y[4 * h + 1]),
                                              __float_as_uint(y[4 * h + 2]), __float_as_uint(y[4 * h + 3])}, dst + h);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        if (v + e < p.V) {
          if constexpr (BF) ((uint16_t*)out)[v + e] = (uint16_t)(pack_bf16x2(y[e], 0.0f) & 0xFFFFu);
          else ((float*)out)[v + e] = y[e];
        }
    }
  }
  wait_vmcnt<0>();  // the columns written over are written
  __syncthreads();
  if (!live) return;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = tid + i * kThreads;
    if (j >= K || ids[j] < 0) continue;
    // the first entry of an id writes its column, with all their weights
    const int64_t id = ids[j];
    bool first = true;
    double q = 0.0;
    for (int k = 0; k < K; ++k)
      if (ids[k] == id) {
        first = first && k >= j;
        q += (double)weights[k];
      }
    if (!first) continue;
    const double pv = exp(((double)own[i] - (double)m) / p.tau) / (double)z;
    const float y = (float)((pv - q) * ((double)p.grad_loss[n] * p.tau));
    if constexpr (BF) ((uint16_t*)out)[id] = (uint16_t)(pack_bf16x2(y, 0.0f) & 0xFFFFu);
    else ((float*)out)[id] = y;
  }
}

int64_t distill_slices(int64_t rows, int64_t V) {
  // enough workgroups to fill the device, of whole turns of their loop
  const int64_t turn = kAhead * kGroup, most = V / turn + (V % turn != 0);
  const int64_t want = rows > 0 && rows < 2048 ? (2048 + rows - 1) / rows : 1;
  const int64_t n = want < most ? want : most;
  return n < 1 ? 1 : n;
}

namespace {
// launch(r0, rows) for parts of the rows whose workgroups fit one launch.
template <typename F>
hipError_t by_rows(int64_t rows, int64_t groups, F launch) {
  const int64_t step = kLaunchGroups / groups;
  if (step < 1) return hipErrorNotSupported;
  for (int64_t r = 0; r < rows; r += step) {
    launch(r, rows - r < step ? rows - r : step);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <bool BF>
hipError_t loss_go(const DistillParams& p, hipStream_t s) {
  const int64_t n = distill_slices(p.rows, p.V);
  const int64_t turn = kAhead * kGroup, slice = ((p.V + n - 1) / n + turn - 1) / turn * turn;
  const int slices = (int)((p.V + slice - 1) / slice);
  hipError_t e = by_rows(p.rows, slices, [&](int64_t r, int64_t rows) {
    hipLaunchKernelGGL(distill_sum_kernel<BF>, dim3((unsigned)(rows * slices)), dim3(kThreads), 0, s, p, r, slices, slice);
  });
  if (e != hipSuccess || slices == 1) return e;
  return by_rows(p.rows, 1, [&](int64_t r, int64_t rows) {
    hipLaunchKernelGGL(distill_finish_kernel<BF>, dim3((unsigned)rows), dim3(kThreads), 0, s, p, r, slices);
  });
}
template <bool BF>
hipError_t backward_go(const DistillParams& p, hipStream_t s) {
  const int64_t slices = (p.V + kBackSlice - 1) / kBackSlice;
  return by_rows(p.rows, slices, [&](int64_t r, int64_t rows) {
    hipLaunchKernelGGL(distill_backward_kernel<BF>, dim3((unsigned)(rows * slices)), dim3(kThreads), 0, s, p, r,
                       (unsigned)slices);
  });
}
}  // namespace

hipError_t launch_distill_loss(const DistillParams& p, bool bf16, hipStream_t s) {
  return bf16 ? loss_go<true>(p, s) : loss_go<false>(p, s);
}

hipError_t launch_distill_backward(const DistillParams& p, bool bf16, hipStream_t s) {
  if (p.K > kDistillMaxEntries) return hipErrorNotSupported;
  return bf16 ? backward_go<true>(p, s) : backward_go<false>(p, s);
}

}  // namespace dspark
