// The global norm of many gradients, and their clipping.
//
//   partials[p] = sum of g^2 over workgroup p's share      (k_grad_norm)
//   norm = sqrt(sum of partials), coef = min(1, max_norm / (norm + 1e-6)),
//   dst = coef * src                                        (k_grad_clip)
//
// The table of tensors lies in device memory. It numbers units of kUnit
// elements through all tensors; a workgroup takes an even, consecutive share
// of the units, looks its first one up once and walks on from there. Squares
// are added in fp64: no gradient overflows them, and the norm of a billion
// values keeps all its fp32 digits. The order of every sum is fixed.
#include "ql_device.h"
#include "ql_ops.h"

namespace ql {

namespace {

typedef __bf16 bf16;
typedef float v4f __attribute__((ext_vector_type(4)));
typedef bf16 v8h __attribute__((ext_vector_type(8)));
typedef bf16 v4h __attribute__((ext_vector_type(4)));
constexpr int kUnit = QL_GRAD_UNIT;
constexpr int kParts = QL_GRAD_PARTIALS;
constexpr int kThreads = 256;

// Last entry whose first unit is <= u (entries are in order): a 64-way search.
__device__ int find_entry(const ql_grad* t, int n, int64_t u) {
  const int lane = threadIdx.x & 63;
  int lo = 0, cnt = n;
  while (cnt > 1) {
    const int step = (cnt + 63) / 64;
    const int i = lane * step;
    const bool le = i < cnt && t[lo + i].start <= u;
    const int k = __popcll(__ballot(le));
    const int at = k > 0 ? (k - 1) * step : 0;
    lo += at;
    cnt = min(step, cnt - at);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  return v;
}

// Sum over the workgroup; valid in every thread.
__device__ double block_sum(double v) {
  __shared__ double w[kThreads / 64];
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) s += w[i];
  return s;
}

__device__ __forceinline__ double sq(double acc, float x) {
  const double d = (double)x;
  return __builtin_fma(d, d, acc);
}

// Sum of squares of p[0 .. n).
__device__ double unit_squares(const float* p, int n) {
  double s0 = 0.0, s1 = 0.0;
  if (n == kUnit && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
    v4f x[kUnit / (4 * kThreads)];
#pragma unroll
    for (int i = 0; i < kUnit / (4 * kThreads); ++i)
      x[i] = reinterpret_cast<const v4f*>(p)[i * kThreads + threadIdx.x];
#pragma unroll
    for (int i = 0; i < kUnit / (4 * kThreads); ++i) {
      s0 = sq(sq(s0, x[i][0]), x[i][1]);
      s1 = sq(sq(s1, x[i][2]), x[i][3]);
    }
  } else {
    for (int i = threadIdx.x; i < n; i += kThreads) s0 = sq(s0, p[i]);
  }
  return s0 + s1;
}
__device__ double unit_squares(const bf16* p, int n) {
  double s0 = 0.0, s1 = 0.0;
  if (n == kUnit && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
    v8h x[kUnit / (8 * kThreads)];
#pragma unroll
    for (int i = 0; i < kUnit / (8 * kThreads); ++i)
      x[i] = reinterpret_cast<const v8h*>(p)[i * kThreads + threadIdx.x];
#pragma unroll
    for (int i = 0; i < kUnit / (8 * kThreads); ++i)
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        s0 = sq(s0, (float)x[i][e]);
        s1 = sq(s1, (float)x[i][e + 1]);
      }
  } else {
    for (int i = threadIdx.x; i < n; i += kThreads) s0 = sq(s0, (float)p[i]);
  }
  return s0 + s1;
}

__global__ __launch_bounds__(kThreads) void k_grad_norm(const ql_grad* t, int n, int64_t units,
                                                        double* partials) {
  const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  double s = 0.0;
  if (u0 < u1 && n > 0) {
    int e = find_entry(t, n, u0);
    for (int64_t u = u0; u < u1; ++u) {
      while (e + 1 < n && t[e + 1].start <= u) ++e;
      const int64_t at = (u - t[e].start) * kUnit;
      if (at < 0 || at >= t[e].n || !t[e].src) continue;
      const int len = (int)min((int64_t)kUnit, t[e].n - at);
      s += t[e].src_dtype == QL_BF16 ? unit_squares(reinterpret_cast<const bf16*>(t[e].src) + at, len)
                                     : unit_squares(reinterpret_cast<const float*>(t[e].src) + at, len);
    }
  }
  s = block_sum(s);
  if (threadIdx.x == 0) partials[blockIdx.x] = s;
  if (blockIdx.x == 0)
    for (int i = gridDim.x + threadIdx.x; i < kParts; i += kThreads) partials[i] = 0.0;
}

template <typename S, typename D>
__device__ void scale_unit(const S* src, D* dst, int n, float c) {
  if (n == kUnit && reinterpret_cast<uintptr_t>(src) % (4 * sizeof(S)) == 0 &&
      reinterpret_cast<uintptr_t>(dst) % (4 * sizeof(D)) == 0) {
    typedef S vs __attribute__((ext_vector_type(4)));
    typedef D vd __attribute__((ext_vector_type(4)));
    vs x[kUnit / (4 * kThreads)];
#pragma unroll
    for (int i = 0; i < kUnit / (4 * kThreads); ++i)
      x[i] = reinterpret_cast<const vs*>(src)[i * kThreads + threadIdx.x];
#pragma unroll
    for (int i = 0; i < kUnit / (4 * kThreads); ++i) {
      vd y;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = (D)((float)x[i][e] * c);
      reinterpret_cast<vd*>(dst)[i * kThreads + threadIdx.x] = y;
    }
  } else {
    for (int i = threadIdx.x; i < n; i += kThreads) dst[i] = (D)((float)src[i] * c);
  }
}

__global__ __launch_bounds__(kThreads) void k_grad_clip(const ql_grad* t, int n, int64_t units,
                                                        const double* partials, float max_norm,
                                                        float* norm) {
  double s = 0.0;
  for (int i = threadIdx.x; i < kParts; i += kThreads) s += partials[i];
  s = block_sum(s);
  const double nr = sqrt(s);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)nr;
  const double q = (double)max_norm / (nr + 1e-6);
  const float c = q >= 1.0 ? 1.0f : (float)q;  // a NaN norm gives a NaN factor
  const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  if (u0 >= u1 || n <= 0) return;
  int e = find_entry(t, n, u0);
  for (int64_t u = u0; u < u1; ++u) {
    while (e + 1 < n && t[e + 1].start <= u) ++e;
    const ql_grad g = t[e];
    const int64_t at = (u - g.start) * kUnit;
    if (at < 0 || at >= g.n || !g.src || !g.dst) continue;
    if (c == 1.0f && g.src == g.dst) continue;  // nothing to change
    const int len = (int)min((int64_t)kUnit, g.n - at);
    if (g.src_dtype == QL_BF16) {
      const bf16* src = reinterpret_cast<const bf16*>(g.src) + at;
      if (g.dst_dtype == QL_BF16)
        scale_unit(src, reinterpret_cast<bf16*>(g.dst) + at, len, c);
      else
        scale_unit(src, reinterpret_cast<float*>(g.dst) + at, len, c);
    } else {
      const float* src = reinterpret_cast<const float*>(g.src) + at;
      if (g.dst_dtype == QL_BF16)
        scale_unit(src, reinterpret_cast<bf16*>(g.dst) + at, len, c);
      else
        scale_unit(src, reinterpret_cast<float*>(g.dst) + at, len, c);
    }
  }
}

}  // namespace

hipError_t launch_grad_norm(const ql_grad* table, int n, int64_t units, double* partials,
                            hipStream_t s) {
  const int grid = (int)(units < 1 ? 1 : units < kParts ? units : kParts);
  hipLaunchKernelGGL(k_grad_norm, dim3(grid), dim3(kThreads), 0, s, table, n, units, partials);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const ql_grad* table, int n, int64_t units, const double* partials,
                            float max_norm, float* norm, hipStream_t s) {
  const int grid = (int)(units < 1 ? 1 : units < 2048 ? units : 2048);
  hipLaunchKernelGGL(k_grad_clip, dim3(grid), dim3(kThreads), 0, s, table, n, units, partials,
                     max_norm, norm);
  return hipGetLastError();
}

}  // namespace ql
