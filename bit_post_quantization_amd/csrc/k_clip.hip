// The global norm of many gradients, and their clipping.
//
//   partials[p] = sum of g^2 over workgroup p's share      (k_grad_norm)
//   norm = sqrt(sum of partials), coef = min(1, max_norm / (norm + 1e-6)),
//   dst = coef * src                                        (k_grad_clip)
//
// The table of tensors lies in device memory and numbers units of kUnit elements
// through all tensors. A workgroup takes runs of consecutive units and looks each
// run's first unit up once; a run inside one tensor is loaded whole before any of
// it is used. Runs follow each other through memory in the order of the
// workgroups, so that those at work at one time share a narrow window of it.
// Squares are added in fp64: no gradient overflows them, and the norm of a billion
// values keeps all its fp32 digits. The order of every sum is fixed.
//
// Bound by memory: 446M bf16 gradients clipped into fp32 (892 MB read twice, 1784 MB
// written) take 640 us, 5.6 TB/s, where a large copy reaches 5.4. The look-up of a
// run is a chain of loads, so long lists take long runs.
#include "ql_device.h"
#include "ql_ops.h"

namespace ql {

namespace {

typedef __bf16 bf16;
typedef float v4f __attribute__((ext_vector_type(4)));
typedef bf16 v8h __attribute__((ext_vector_type(8)));
constexpr int kUnit = QL_GRAD_UNIT;
constexpr int kParts = QL_GRAD_PARTIALS;
constexpr int kThreads = 512;

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

// The entry of a run's first unit, and whether the run lies whole inside it.
struct Run {
  int e;
  bool whole;
  int64_t at;  // element of the entry at which the run starts
};
__device__ __forceinline__ Run find_run(const ql_grad* t, int n, int64_t u, int units) {
  Run r;
  r.e = find_entry(t, n, u);
  r.at = (u - t[r.e].start) * kUnit;
  r.whole = r.at >= 0 && t[r.e].src && r.at + (int64_t)units * kUnit <= t[r.e].n;
  return r;
}

// Sum of squares of R whole units from p on.
template <int R>
__device__ __forceinline__ double run_squares(const float* p) {
  constexpr int N = R * kUnit / (4 * kThreads);
  v4f x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = reinterpret_cast<const v4f*>(p)[i * kThreads + threadIdx.x];
  double s0 = 0.0, s1 = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s0 = sq(sq(s0, x[i][0]), x[i][1]);
    s1 = sq(sq(s1, x[i][2]), x[i][3]);
  }
  return s0 + s1;
}
template <int R>
__device__ __forceinline__ double run_squares(const bf16* p) {
  constexpr int N = R * kUnit / (8 * kThreads);
  v8h x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = reinterpret_cast<const v8h*>(p)[i * kThreads + threadIdx.x];
  double s0 = 0.0, s1 = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      s0 = sq(s0, (float)x[i][e]);
      s1 = sq(s1, (float)x[i][e + 1]);
    }
  return s0 + s1;
}
// Of one unit of n <= kUnit elements, at any alignment.
template <typename T>
__device__ __forceinline__ double part_squares(const T* p, int n) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s = sq(s, (float)p[i]);
  return s;
}

template <int R, typename T>
__device__ __forceinline__ double squares(const void* src, int64_t at) {
  return run_squares<R>(reinterpret_cast<const T*>(src) + at);
}

template <int R>
__global__ __launch_bounds__(kThreads) void k_grad_norm(const ql_grad* t, int n, int64_t units,
                                                        double* partials) {
  double s = 0.0;
  for (int64_t u0 = (int64_t)blockIdx.x * R; u0 < units; u0 += (int64_t)gridDim.x * R) {
    const Run r = find_run(t, n, u0, R);
    if (r.whole && reinterpret_cast<uintptr_t>(t[r.e].src) % 16 == 0) {
      s += t[r.e].src_dtype == QL_BF16 ? squares<R, bf16>(t[r.e].src, r.at)
                                       : squares<R, float>(t[r.e].src, r.at);
      continue;
    }
    int e = r.e;
    for (int64_t u = u0; u < min(u0 + R, units); ++u) {
      while (e + 1 < n && t[e + 1].start <= u) ++e;
      const int64_t at = (u - t[e].start) * kUnit;
      if (at < 0 || at >= t[e].n || !t[e].src) continue;
      const int len = (int)min((int64_t)kUnit, t[e].n - at);
      const bool vec = len == kUnit && reinterpret_cast<uintptr_t>(t[e].src) % 16 == 0;
      if (t[e].src_dtype == QL_BF16)
        s += vec ? squares<1, bf16>(t[e].src, at)
                 : part_squares(reinterpret_cast<const bf16*>(t[e].src) + at, len);
      else
        s += vec ? squares<1, float>(t[e].src, at)
                 : part_squares(reinterpret_cast<const float*>(t[e].src) + at, len);
    }
  }
  s = block_sum(s);
  if (threadIdx.x == 0) partials[blockIdx.x] = s;
  if (blockIdx.x == 0)
    for (int i = gridDim.x + threadIdx.x; i < kParts; i += kThreads) partials[i] = 0.0;
}

// The factor, from the partial sums; the first workgroup writes the norm. A NaN
// norm gives a NaN factor.
__device__ __forceinline__ float clip_factor(const double* partials, float max_norm, float* norm) {
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kParts / kThreads; ++i) s += partials[i * kThreads + threadIdx.x];
  const double nr = sqrt(block_sum(s));
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)nr;
  const double q = (double)max_norm / (nr + 1e-6);
  return q >= 1.0 ? 1.0f : (float)q;
}

// R whole units: the loads first, then the factor, which the loads do not wait for.
template <int R, typename S, typename D, typename F>
__device__ __forceinline__ void scale_run(const S* src, D* dst, bool in_place, F factor) {
  constexpr int N = R * kUnit / (4 * kThreads);
  typedef S vs __attribute__((ext_vector_type(4)));
  typedef D vd __attribute__((ext_vector_type(4)));
  vs x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = reinterpret_cast<const vs*>(src)[i * kThreads + threadIdx.x];
  const float c = factor();
  if (c == 1.0f && in_place) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    vd y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = (D)((float)x[i][e] * c);
    reinterpret_cast<vd*>(dst)[i * kThreads + threadIdx.x] = y;
  }
}
template <typename S, typename D>
__device__ __forceinline__ void scale_part(const S* src, D* dst, int n, float c) {
  for (int i = threadIdx.x; i < n; i += kThreads) dst[i] = (D)((float)src[i] * c);
}

template <int R, typename F>
__device__ __forceinline__ void scale_any(const ql_grad& g, int64_t at, int len, F factor) {
  // len == R * kUnit and aligned: whole; else one short or unaligned unit
  const bool in_place = g.src == g.dst;
  auto go = [&](auto* src, auto* dst) {
    const bool vec = len == R * kUnit && reinterpret_cast<uintptr_t>(src) % (4 * sizeof(*src)) == 0 &&
                     reinterpret_cast<uintptr_t>(dst) % (4 * sizeof(*dst)) == 0;
    if (vec) {
      scale_run<R>(src + at, dst + at, in_place, factor);
    } else {
      const float c = factor();
      if (c == 1.0f && in_place) return;
      scale_part(src + at, dst + at, len, c);
    }
  };
  if (g.src_dtype == QL_BF16) {
    const bf16* src = reinterpret_cast<const bf16*>(g.src);
    if (g.dst_dtype == QL_BF16)
      go(src, reinterpret_cast<bf16*>(g.dst));
    else
      go(src, reinterpret_cast<float*>(g.dst));
  } else {
    const float* src = reinterpret_cast<const float*>(g.src);
    if (g.dst_dtype == QL_BF16)
      go(src, reinterpret_cast<bf16*>(g.dst));
    else
      go(src, reinterpret_cast<float*>(g.dst));
  }
}

template <int R>
__global__ __launch_bounds__(kThreads) void k_grad_clip(const ql_grad* t, int n, int64_t units,
                                                        const double* partials, float max_norm,
                                                        float* norm) {
  bool known = false;
  float c = 0.0f;
  auto factor = [&]() {
    if (!known) c = clip_factor(partials, max_norm, norm);
    known = true;
    return c;
  };
  for (int64_t u0 = (int64_t)blockIdx.x * R; u0 < units; u0 += (int64_t)gridDim.x * R) {
    const Run r = find_run(t, n, u0, R);
    const ql_grad g = t[r.e];
    if (r.whole && g.dst) {
      scale_any<R>(g, r.at, R * kUnit, factor);
      continue;
    }
    int e = r.e;
    for (int64_t u = u0; u < min(u0 + R, units); ++u) {
      while (e + 1 < n && t[e + 1].start <= u) ++e;
      const ql_grad h = t[e];
      const int64_t at = (u - h.start) * kUnit;
      if (at < 0 || at >= h.n || !h.src || !h.dst) continue;
      scale_any<1>(h, at, (int)min((int64_t)kUnit, h.n - at), factor);
    }
  }
  factor();  // without a unit of its own the first workgroup still writes the norm
}

// Units of a run. With runs of one / four: 3.3M fp32 gradients 10.2 / 13.3 us, 8.3M
// (224 adapter tensors) 27.2 / 28.4 us, 33M 80 / 84 us; 446M bf16 ones 1001 / 645 us.
int run_units(int64_t units) { return units >= 16384 ? 4 : 1; }

}  // namespace

hipError_t launch_grad_norm(const ql_grad* table, int n, int64_t units, double* partials,
                            hipStream_t s) {
  const int run = run_units(units);
  const int64_t runs = (units + run - 1) / run;
  const dim3 grid((unsigned)(runs < 1 ? 1 : runs < kParts ? runs : kParts)), block(kThreads);
  if (run == 4)
    hipLaunchKernelGGL(k_grad_norm<4>, grid, block, 0, s, table, n, units, partials);
  else
    hipLaunchKernelGGL(k_grad_norm<1>, grid, block, 0, s, table, n, units, partials);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const ql_grad* table, int n, int64_t units, const double* partials,
                            float max_norm, float* norm, hipStream_t s) {
  const int run = run_units(units);
  const int64_t runs = (units + run - 1) / run, most = 1 << 20;
  const dim3 grid((unsigned)(runs < 1 ? 1 : runs < most ? runs : most)), block(kThreads);
  if (run == 4)
    hipLaunchKernelGGL(k_grad_clip<4>, grid, block, 0, s, table, n, units, partials, max_norm, norm);
  else
    hipLaunchKernelGGL(k_grad_clip<1>, grid, block, 0, s, table, n, units, partials, max_norm, norm);
  return hipGetLastError();
}

}  // namespace ql
