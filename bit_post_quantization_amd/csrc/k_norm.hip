// Group normalisation with an activation over channels-last images.
//
//   forward   z = (x - mean_g) rstd_g gamma_c + beta_c,  y = act(z)
//   backward  dz = dy act'(z); dbeta_c = sum dz; dgamma_c = sum dz xhat;
//             dx = rstd (dz gamma - s1 - xhat s2), s1 / s2 the group's means
//             of dz gamma and dz gamma xhat
//
// Both directions read their inputs in chunks of positions. A thread keeps the
// same channels for all its positions, so a channel's sums stay in registers;
// they are joined in a fixed order (LDS, then the chunks), with no atomics.
// Sums of x and x^2 are kept as shifted fp32 sums inside a thread (the shift is
// the thread's first value of the channel) and in fp64 beyond it, so a mean
// far from zero costs no digits of the variance.
#include "ql_device.h"
#include "ql_ops.h"

namespace ql {

namespace {

typedef __bf16 bf16;
constexpr int kNormThreads = 512;
constexpr float kLog2e = 1.44269504088896340736f;

template <typename T, int V>
struct Vec {
  typedef T type __attribute__((ext_vector_type(V)));
};
template <typename T>
struct Vec<T, 1> {
  typedef T type;
};

template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = (float)p[0];
  } else {
    const typename Vec<T, V>::type x = *reinterpret_cast<const typename Vec<T, V>::type*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (float)x[i];
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    p[0] = (T)v[0];
  } else {
    typename Vec<T, V>::type x;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = (T)v[i];
    *reinterpret_cast<typename Vec<T, V>::type*>(p) = x;
  }
}

// 1 / (1 + exp(-z)): exp from the hardware's base-2 exponential, relative
// error about |z| 2^-24; the reciprocal is within one unit in the last place.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
}

// Position p of image b is chunk-local; thread (tx, ty) of a workgroup takes
// channel vectors tx, tx + TX, ... of positions ty, ty + TY, ...
struct Shape {
  int B, L, C, G, cpg, cv, tx, ty, chunks, rows;  // rows: positions of a chunk
};

struct StatsK {
  const void* x;
  int64_t xb, xr;
  double2* part;  // [B][chunks][G]: sum, sum of squares
  Shape s;
};

template <typename T, int V>
__global__ __launch_bounds__(kNormThreads) void k_norm_stats(StatsK a) {
  extern __shared__ float2 lds2[];  // [TY][C]: mean, M2 of a thread's channel
  const Shape& s = a.s;
  const int tx = threadIdx.x % s.tx, ty = threadIdx.x / s.tx;
  const int b = blockIdx.y, chunk = blockIdx.x;
  const int l0 = chunk * s.rows, l1 = min(s.L, l0 + s.rows);
  const T* x = reinterpret_cast<const T*>(a.x) + b * a.xb;
  if (ty < s.ty) {
    for (int v = tx; v < s.cv; v += s.tx) {
      float k[V], s1[V], s2[V];
#pragma unroll
      for (int i = 0; i < V; ++i) k[i] = s1[i] = s2[i] = 0.0f;
      if (l0 + ty < l1) load_v<T, V>(x + (int64_t)(l0 + ty) * a.xr + v * V, k);
      int n = 0;
      for (int l = l0 + ty; l < l1; l += s.ty, ++n) {
        float e[V];
        load_v<T, V>(x + (int64_t)l * a.xr + v * V, e);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float d = e[i] - k[i];
          s1[i] += d;
          s2[i] = __builtin_fmaf(d, d, s2[i]);
        }
      }
      const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float md = s1[i] * inv;
        lds2[ty * s.C + v * V + i] = float2{k[i] + md, s2[i] - s1[i] * md};
      }
    }
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, nw = blockDim.x >> 6;
  for (int g = threadIdx.x >> 6; g < s.G; g += nw) {
    double S = 0.0, Q = 0.0;
    for (int e = lane; e < s.ty * s.cpg; e += kWave) {
      const int y = e / s.cpg, c = g * s.cpg + e % s.cpg;
      const int n = l0 + y < l1 ? (l1 - l0 - y + s.ty - 1) / s.ty : 0;
      const float2 m = lds2[y * s.C + c];
      if (n > 0) {
        S += (double)n * m.x;
        Q += (double)m.y + (double)n * m.x * m.x;
      }
    }
#pragma unroll
    for (int d = kWave / 2; d > 0; d /= 2) {
      S += __shfl_xor(S, d);
      Q += __shfl_xor(Q, d);
    }
    if (lane == 0) a.part[((int64_t)b * s.chunks + chunk) * s.G + g] = double2{S, Q};
  }
}

struct ApplyK {
  const void* x;
  int64_t xb, xr;
  void* y;
  int64_t yb, yr;
  const void* gamma;
  const void* beta;
  const double2* part;
  float* mean;
  float* rstd;
  float eps;
  Shape s;
};

template <typename T, typename W, int V, bool SILU>
__global__ __launch_bounds__(kNormThreads) void k_norm_apply(ApplyK a) {
  extern __shared__ float2 lds2[];  // [G]: mean, rstd
  __shared__ double2 sub[kNormThreads];
  const Shape& s = a.s;
  const int b = blockIdx.y, chunk = blockIdx.x;
  {
    const int gb = min(s.G, (int)blockDim.x), ns = blockDim.x / gb;
    const int gi = threadIdx.x % gb, si = threadIdx.x / gb;
    for (int g0 = 0; g0 < s.G; g0 += gb) {
      double S = 0.0, Q = 0.0;
      const int g = g0 + gi;
      if (si < ns && g < s.G) {
        const double2* p = a.part + (int64_t)b * s.chunks * s.G + g;
        for (int c = si; c < s.chunks; c += ns) {
          S += p[(int64_t)c * s.G].x;
          Q += p[(int64_t)c * s.G].y;
        }
      }
      sub[threadIdx.x] = double2{S, Q};
      __syncthreads();
      if (si == 0 && g < s.G) {
        for (int u = 1; u < ns; ++u) {
          S += sub[u * gb + gi].x;
          Q += sub[u * gb + gi].y;
        }
        const double n = (double)s.L * s.cpg, m = S / n, var = fmax(Q / n - m * m, 0.0);
        const float2 r{(float)m, (float)(1.0 / sqrt(var + (double)a.eps))};
        lds2[g] = r;
        if (chunk == 0) {
          if (a.mean) a.mean[b * s.G + g] = r.x;
          if (a.rstd) a.rstd[b * s.G + g] = r.y;
        }
      }
      __syncthreads();
    }
  }
  const int tx = threadIdx.x % s.tx, ty = threadIdx.x / s.tx;
  if (ty >= s.ty) return;
  const int l0 = chunk * s.rows, l1 = min(s.L, l0 + s.rows);
  const T* x = reinterpret_cast<const T*>(a.x) + b * a.xb;
  T* y = reinterpret_cast<T*>(a.y) + b * a.yb;
  const W* gamma = reinterpret_cast<const W*>(a.gamma);
  const W* beta = reinterpret_cast<const W*>(a.beta);
  for (int v = tx; v < s.cv; v += s.tx) {
    float m[V], sc[V], sh[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = v * V + i;
      const float2 r = lds2[c / s.cpg];
      m[i] = r.x;
      sc[i] = r.y * (gamma ? (float)gamma[c] : 1.0f);
      sh[i] = beta ? (float)beta[c] : 0.0f;
    }
    for (int l = l0 + ty; l < l1; l += s.ty) {
      float e[V];
      load_v<T, V>(x + (int64_t)l * a.xr + v * V, e);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float z = __builtin_fmaf(e[i] - m[i], sc[i], sh[i]);
        e[i] = SILU ? z * sigmoid(z) : z;
      }
      store_v<T, V>(y + (int64_t)l * a.yr + v * V, e);
    }
  }
}

struct GradK {
  const void* x;
  int64_t xb, xr;
  const void* dy;
  int64_t dyb, dyr;
  void* dx;
  int64_t dxb, dxr;
  const void* gamma;
  const void* beta;
  const float* mean;
  const float* rstd;
  float2* part;  // [B][chunks][C]: sum dz, sum dz xhat over a chunk
  float2* pq;    // [B][C]
  float2* s12;   // [B][G]
  void* dgamma;
  void* dbeta;
  Shape s;
};

// dz of one value; xh receives xhat.
template <bool SILU>
__device__ __forceinline__ float grad_z(float x, float dy, float m, float r, float ga, float be,
                                        float& xh) {
  xh = (x - m) * r;
  if constexpr (!SILU) return dy;
  const float z = __builtin_fmaf(xh, ga, be);
  const float sg = sigmoid(z);
  return dy * (sg * __builtin_fmaf(z, 1.0f - sg, 1.0f));
}

template <typename T, typename W, int V, bool SILU>
__global__ __launch_bounds__(kNormThreads) void k_norm_grad_sums(GradK a) {
  extern __shared__ float2 lds2[];  // [TY][C]
  const Shape& s = a.s;
  const int tx = threadIdx.x % s.tx, ty = threadIdx.x / s.tx;
  const int b = blockIdx.y, chunk = blockIdx.x;
  const int l0 = chunk * s.rows, l1 = min(s.L, l0 + s.rows);
  const T* x = reinterpret_cast<const T*>(a.x) + b * a.xb;
  const T* dy = reinterpret_cast<const T*>(a.dy) + b * a.dyb;
  const W* gamma = reinterpret_cast<const W*>(a.gamma);
  const W* beta = reinterpret_cast<const W*>(a.beta);
  if (ty < s.ty) {
    for (int v = tx; v < s.cv; v += s.tx) {
      float m[V], r[V], ga[V], be[V], p[V], q[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = v * V + i, g = b * s.G + c / s.cpg;
        m[i] = a.mean[g];
        r[i] = a.rstd[g];
        ga[i] = gamma ? (float)gamma[c] : 1.0f;
        be[i] = beta ? (float)beta[c] : 0.0f;
        p[i] = q[i] = 0.0f;
      }
      for (int l = l0 + ty; l < l1; l += s.ty) {
        float e[V], d[V];
        load_v<T, V>(x + (int64_t)l * a.xr + v * V, e);
        load_v<T, V>(dy + (int64_t)l * a.dyr + v * V, d);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float xh;
          const float dz = grad_z<SILU>(e[i], d[i], m[i], r[i], ga[i], be[i], xh);
          p[i] += dz;
          q[i] = __builtin_fmaf(dz, xh, q[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) lds2[ty * s.C + v * V + i] = float2{p[i], q[i]};
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < s.C; c += blockDim.x) {
    float p = 0.0f, q = 0.0f;
    for (int y = 0; y < s.ty; ++y) {
      p += lds2[y * s.C + c].x;
      q += lds2[y * s.C + c].y;
    }
    a.part[((int64_t)b * s.chunks + chunk) * s.C + c] = float2{p, q};
  }
}

// One workgroup per image and group: the chunks of its channels, then the
// group's two means.
template <typename W>
__global__ __launch_bounds__(256) void k_norm_grad_reduce(GradK a) {
  __shared__ double2 sub[256];
  const Shape& s = a.s;
  const int b = blockIdx.x / s.G, g = blockIdx.x % s.G;
  const W* gamma = reinterpret_cast<const W*>(a.gamma);
  const int cb = min(s.cpg, 256), ns = 256 / cb;
  const int ci = threadIdx.x % cb, si = threadIdx.x / cb;
  double s1 = 0.0, s2 = 0.0;
  for (int c0 = 0; c0 < s.cpg; c0 += cb) {
    const int c = g * s.cpg + c0 + ci;
    const bool live = si < ns && c0 + ci < s.cpg;
    double P = 0.0, Q = 0.0;
    if (live) {
      for (int k = si; k < s.chunks; k += ns) {
        const float2 v = a.part[((int64_t)b * s.chunks + k) * s.C + c];
        P += v.x;
        Q += v.y;
      }
    }
    sub[threadIdx.x] = double2{P, Q};
    __syncthreads();
    if (live && si == 0) {
      for (int u = 1; u < ns; ++u) {
        P += sub[u * cb + ci].x;
        Q += sub[u * cb + ci].y;
      }
      a.pq[(int64_t)b * s.C + c] = float2{(float)P, (float)Q};
      const double ga = gamma ? (double)(float)gamma[c] : 1.0;
      s1 += ga * P;
      s2 += ga * Q;
    }
    __syncthreads();
  }
  sub[threadIdx.x] = double2{s1, s2};
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int u = 1; u < cb; ++u) {
      s1 += sub[u].x;
      s2 += sub[u].y;
    }
    const double n = (double)s.L * s.cpg;
    a.s12[b * s.G + g] = float2{(float)(s1 / n), (float)(s2 / n)};
  }
}

template <typename T, typename W, int V, bool SILU>
__global__ __launch_bounds__(kNormThreads) void k_norm_grad_apply(GradK a) {
  const Shape& s = a.s;
  if ((int)blockIdx.x >= s.chunks) {  // dgamma and dbeta: sums over the images
    const int c = ((int)blockIdx.x - s.chunks) * kNormThreads + threadIdx.x;
    if (blockIdx.y != 0 || c >= s.C) return;
    double p = 0.0, q = 0.0;
    for (int b = 0; b < s.B; ++b) {
      const float2 v = a.pq[(int64_t)b * s.C + c];
      p += v.x;
      q += v.y;
    }
    if (a.dgamma) reinterpret_cast<W*>(a.dgamma)[c] = (W)(float)q;
    if (a.dbeta) reinterpret_cast<W*>(a.dbeta)[c] = (W)(float)p;
    return;
  }
  const int tx = threadIdx.x % s.tx, ty = threadIdx.x / s.tx;
  if (ty >= s.ty) return;
  const int b = blockIdx.y, chunk = blockIdx.x;
  const int l0 = chunk * s.rows, l1 = min(s.L, l0 + s.rows);
  const T* x = reinterpret_cast<const T*>(a.x) + b * a.xb;
  const T* dy = reinterpret_cast<const T*>(a.dy) + b * a.dyb;
  T* dx = reinterpret_cast<T*>(a.dx) + b * a.dxb;
  const W* gamma = reinterpret_cast<const W*>(a.gamma);
  const W* beta = reinterpret_cast<const W*>(a.beta);
  for (int v = tx; v < s.cv; v += s.tx) {
    float m[V], r[V], ga[V], be[V], s1[V], s2[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = v * V + i, g = b * s.G + c / s.cpg;
      m[i] = a.mean[g];
      r[i] = a.rstd[g];
      ga[i] = gamma ? (float)gamma[c] : 1.0f;
      be[i] = beta ? (float)beta[c] : 0.0f;
      const float2 t = a.s12[g];
      s1[i] = t.x;
      s2[i] = t.y;
    }
    for (int l = l0 + ty; l < l1; l += s.ty) {
      float e[V], d[V];
      load_v<T, V>(x + (int64_t)l * a.xr + v * V, e);
      load_v<T, V>(dy + (int64_t)l * a.dyr + v * V, d);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float xh;
        const float dz = grad_z<SILU>(e[i], d[i], m[i], r[i], ga[i], be[i], xh);
        e[i] = r[i] * (dz * ga[i] - s1[i] - xh * s2[i]);
      }
      store_v<T, V>(dx + (int64_t)l * a.dxr + v * V, e);
    }
  }
}

// Elements that one access may cover: 16 bytes where every row starts aligned
// and C divides, else one element.
bool rows_aligned(const void* p, int64_t sb, int64_t sr, int es) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (sb * es) % 16 == 0 && (sr * es) % 16 == 0;
}

Shape shape_of(int B, int L, int C, int G, int V) {
  Shape s;
  s.B = B;
  s.L = L;
  s.C = C;
  s.G = G;
  s.cpg = C / G;
  s.cv = C / V;
  s.tx = s.cv < kNormThreads ? s.cv : kNormThreads;
  s.ty = kNormThreads / s.tx;
  // About 1024 workgroups in all, none with fewer positions than it has rows
  // of threads.
  int64_t want = (1024 + B - 1) / B;
  const int64_t cap = (L + s.ty - 1) / s.ty;
  want = want < cap ? want : cap;
  s.rows = (int)(((int64_t)L + want - 1) / want);
  s.rows = (s.rows + s.ty - 1) / s.ty * s.ty;
  s.chunks = (L + s.rows - 1) / s.rows;
  return s;
}

template <typename T, typename W, int V>
hipError_t norm_run(const NormArgs& a, hipStream_t st) {
  const Shape s = shape_of(a.B, a.L, a.C, a.G, V);
  double2* part = reinterpret_cast<double2*>(a.ws);
  const int threads = (s.tx * s.ty + 63) / 64 * 64;
  hipLaunchKernelGGL((k_norm_stats<T, V>), dim3(s.chunks, s.B), dim3(threads),
                     (size_t)s.ty * s.C * sizeof(float2), st, StatsK{a.x, a.xb, a.xr, part, s});
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const ApplyK k{a.x, a.xb, a.xr, a.y, a.yb, a.yr, a.gamma, a.beta, part, a.mean, a.rstd, a.eps, s};
  const size_t lds = (size_t)s.G * sizeof(float2);
  if (a.act)
    hipLaunchKernelGGL((k_norm_apply<T, W, V, true>), dim3(s.chunks, s.B), dim3(threads), lds, st, k);
  else
    hipLaunchKernelGGL((k_norm_apply<T, W, V, false>), dim3(s.chunks, s.B), dim3(threads), lds, st,
                       k);
  return hipGetLastError();
}

template <typename T, typename W, int V>
hipError_t norm_grad_run(const NormArgs& a, hipStream_t st) {
  const bool empty = a.B == 0 || a.L == 0;  // dgamma and dbeta are still written: zero
  Shape s = shape_of(empty ? 1 : a.B, empty ? 1 : a.L, a.C, a.G, V);
  if (empty) s.B = s.chunks = 0;
  float2* pq = reinterpret_cast<float2*>(a.ws);
  float2* s12 = pq + (int64_t)s.B * s.C;
  float2* part = s12 + (int64_t)s.B * s.G;
  const GradK k{a.x,     a.xb,    a.xr, a.dy, a.dyb, a.dyr, a.y,      a.yb,    a.yr, a.gamma, a.beta,
                a.mean, a.rstd, part, pq,   s12,   a.dgamma, a.dbeta, s};
  const int threads = (s.tx * s.ty + 63) / 64 * 64;
  const size_t lds = (size_t)s.ty * s.C * sizeof(float2);
  if (!empty) {
    if (a.act)
      hipLaunchKernelGGL((k_norm_grad_sums<T, W, V, true>), dim3(s.chunks, s.B), dim3(threads), lds,
                         st, k);
    else
      hipLaunchKernelGGL((k_norm_grad_sums<T, W, V, false>), dim3(s.chunks, s.B), dim3(threads),
                         lds, st, k);
    hipLaunchKernelGGL(k_norm_grad_reduce<W>, dim3(s.B * s.G), dim3(256), 0, st, k);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid(s.chunks + (s.C + kNormThreads - 1) / kNormThreads, empty ? 1 : s.B);
  if (a.act)
    hipLaunchKernelGGL((k_norm_grad_apply<T, W, V, true>), grid, dim3(kNormThreads), 0, st, k);
  else
    hipLaunchKernelGGL((k_norm_grad_apply<T, W, V, false>), grid, dim3(kNormThreads), 0, st, k);
  return hipGetLastError();
}

template <typename T, typename W>
hipError_t norm_dispatch(const NormArgs& a, bool grad, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const int es = sizeof(T);
  const bool vec = a.C % V == 0 && rows_aligned(a.x, a.xb, a.xr, es) &&
                   rows_aligned(a.y, a.yb, a.yr, es) &&
                   (!grad || rows_aligned(a.dy, a.dyb, a.dyr, es));
  if (grad) return vec ? norm_grad_run<T, W, V>(a, st) : norm_grad_run<T, W, 1>(a, st);
  return vec ? norm_run<T, W, V>(a, st) : norm_run<T, W, 1>(a, st);
}

hipError_t norm_types(const NormArgs& a, bool grad, hipStream_t s) {
  if (a.x_bf16)
    return a.w_bf16 ? norm_dispatch<bf16, bf16>(a, grad, s) : norm_dispatch<bf16, float>(a, grad, s);
  return a.w_bf16 ? norm_dispatch<float, bf16>(a, grad, s) : norm_dispatch<float, float>(a, grad, s);
}

}  // namespace

int64_t norm_ws_bytes(int B, int L, int C, int G, bool grad) {
  int64_t chunks = 0;  // the most of any vector width
  for (int V : {1, 4, 8}) {
    if (C % V) continue;
    const Shape s = shape_of(B, L, C, G, V);
    chunks = chunks > s.chunks ? chunks : s.chunks;
  }
  if (!grad) return (int64_t)B * chunks * G * (int64_t)sizeof(double2);
  return ((int64_t)B * C + (int64_t)B * G + (int64_t)B * chunks * C) * (int64_t)sizeof(float2);
}

hipError_t launch_group_norm(const NormArgs& a, hipStream_t s) { return norm_types(a, false, s); }

hipError_t launch_group_norm_grad(const NormArgs& a, hipStream_t s) {
  return norm_types(a, true, s);
}

}  // namespace ql
