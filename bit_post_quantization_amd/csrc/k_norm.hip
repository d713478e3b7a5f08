// Group normalisation with an activation over channels-last images.
//
//   forward   z = (x - mean_g) rstd_g gamma_c + beta_c,  y = act(z)
//   backward  dz = dy act'(z); dbeta_c = sum dz; dgamma_c = sum dz xhat;
//             dx = rstd (dz gamma - s1 - xhat s2), s1 / s2 the group's means
//             of dz gamma and dz gamma xhat
//
// Where one image's group (its slab) fits a workgroup's registers, one workgroup
// takes it whole: everything is read once and written once, in one launch
// (k_norm_slab, k_norm_slab_grad). Otherwise the inputs are read twice, in chunks
// of positions: sums, their joining, then the result (the second reading mostly
// comes from the chip's last-level cache). A thread keeps the same channels for
// all its positions, four positions' loads in flight; sums are joined in a fixed
// order, with no atomics.
//
// Sums of x are taken about a value of x (the thread's or the slab's first) and
// joined in fp64, or squares are taken about the mean itself, so a mean far from
// zero costs no digits of the variance.
//
// Measured per call (MI355X; a copy of the bytes read and written once in brackets):
//   2x256x1280 bf16: 6.5 us of kernel, 7.7 us a call; latency: load, two sums over the
//     workgroup, store
//   8x16384x320 bf16 (84 MB): 65 us (31): 17 us of sums at 4.9 TB/s, 4.5 of joining
//     them, 33 of writing at 5.1 TB/s, read again from the last-level cache, and 10
//     between the three launches
//   gradient of 4x1024x640 fp32 (31 MB): 16.4 us (6): 128 slabs for 256 compute units,
//     bound by the arithmetic of a SiLU's gradient
//   gradient of 4x16383x256 bf16 (101 MB): 46 us (19): 17 us of sums, 4 of joining them
//     and 26 of writing, 4.0 TB/s
#include "ql_device.h"
#include "ql_ops.h"

namespace ql {

namespace {

typedef __bf16 bf16;
constexpr int kNormThreads = 512;
// Vectors of a slab that a thread holds at most: 192 bytes, 48 vectors.
constexpr int slab_most(int bytes) { return 192 / bytes < 48 ? 192 / bytes : 48; }
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
__device__ __forceinline__ typename Vec<T, V>::type raw_v(const T* p) {
  return *reinterpret_cast<const typename Vec<T, V>::type*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void widen(const typename Vec<T, V>::type& x, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = (float)x;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (float)x[i];
  }
}
template <typename T, int V>
__device__ __forceinline__ void put_v(typename Vec<T, V>::type& x, int i, float v) {
  if constexpr (V == 1)
    x = (T)v;
  else
    x[i] = (T)v;
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

template <bool SILU>
__device__ __forceinline__ float act(float z) {
  return SILU ? z * sigmoid(z) : z;
}

// gamma and beta of V channels from c on (1 and 0 where there is none).
template <typename W, int V>
struct Affine {
  float ga[V], be[V];
  __device__ __forceinline__ void load(const void* gamma, const void* beta, int c) {
    const W* g = reinterpret_cast<const W*>(gamma);
    const W* b = reinterpret_cast<const W*>(beta);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ga[i] = g ? (float)g[c + i] : 1.0f;
      be[i] = b ? (float)b[c + i] : 0.0f;
    }
  }
};

// A variance that roundings took below zero is zero; a NaN stays one (fmax would drop it).
__device__ __forceinline__ double variance(double v) { return v < 0.0 ? 0.0 : v; }

constexpr int kAhead = 4;  // positions whose loads a thread has in flight

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
      const T* p = x + v * V;
      int n = 0;
      auto add = [&](const typename Vec<T, V>::type& xv) {
        float e[V];
        widen<T, V>(xv, e);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (n == 0) k[i] = e[i];
          const float d = e[i] - k[i];
          s1[i] += d;
          s2[i] = __builtin_fmaf(d, d, s2[i]);
        }
        ++n;
      };
      int l = l0 + ty;
      for (; l + (kAhead - 1) * s.ty < l1; l += kAhead * s.ty) {
        typename Vec<T, V>::type e[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) e[j] = raw_v<T, V>(p + (int64_t)(l + j * s.ty) * a.xr);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) add(e[j]);
      }
      for (; l < l1; l += s.ty) add(raw_v<T, V>(p + (int64_t)l * a.xr));
      const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float md = s1[i] * inv;
        // in fp64, so that squares past fp32 stay infinite and are not inf - inf
        const double m2 = (double)s2[i] - (double)s1[i] * (double)md;
        lds2[ty * s.C + v * V + i] = float2{k[i] + md, (float)m2};
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

// mean and rstd of every image's group from its chunks: one wave a group.
struct StatsOut {
  float2* stats;  // [B][G]: mean, rstd; or nullptr
  float* mean;    // the caller's, or nullptr
  float* rstd;
  float eps;
};

__global__ __launch_bounds__(256) void k_norm_stats_join(const double2* part, StatsOut o, Shape s) {
  const int lane = threadIdx.x & 63, id = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (id >= s.B * s.G) return;
  const int b = id / s.G, g = id % s.G;
  double S = 0.0, Q = 0.0;
  for (int c = lane; c < s.chunks; c += kWave) {
    const double2 v = part[((int64_t)b * s.chunks + c) * s.G + g];
    S += v.x;
    Q += v.y;
  }
#pragma unroll
  for (int d = kWave / 2; d > 0; d /= 2) {
    S += __shfl_xor(S, d);
    Q += __shfl_xor(Q, d);
  }
  if (lane != 0) return;
  const double n = (double)s.L * s.cpg, m = S / n, var = variance(Q / n - m * m);
  const float2 r{(float)m, (float)(1.0 / sqrt(var + (double)o.eps))};
  if (o.stats) o.stats[id] = r;
  if (o.mean) o.mean[id] = r.x;
  if (o.rstd) o.rstd[id] = r.y;
}

struct ApplyK {
  const void* x;
  int64_t xb, xr;
  void* y;
  int64_t yb, yr;
  const void* gamma;
  const void* beta;
  const float2* stats;
  Shape s;
};

template <typename T, typename W, int V, bool SILU>
__global__ __launch_bounds__(kNormThreads) void k_norm_apply(ApplyK a) {
  const Shape& s = a.s;
  const int b = blockIdx.y, chunk = blockIdx.x;
  const int tx = threadIdx.x % s.tx, ty = threadIdx.x / s.tx;
  if (ty >= s.ty) return;
  const int l0 = chunk * s.rows, l1 = min(s.L, l0 + s.rows);
  const T* x = reinterpret_cast<const T*>(a.x) + b * a.xb;
  T* y = reinterpret_cast<T*>(a.y) + b * a.yb;
  for (int v = tx; v < s.cv; v += s.tx) {
    Affine<W, V> f;
    f.load(a.gamma, a.beta, v * V);
    float m[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 r = a.stats[b * s.G + (v * V + i) / s.cpg];
      m[i] = r.x;
      f.ga[i] *= r.y;
    }
    auto put = [&](const typename Vec<T, V>::type& xv, int l) {
      float e[V];
      widen<T, V>(xv, e);
#pragma unroll
      for (int i = 0; i < V; ++i) e[i] = act<SILU>(__builtin_fmaf(e[i] - m[i], f.ga[i], f.be[i]));
      store_v<T, V>(y + (int64_t)l * a.yr + v * V, e);
    };
    const T* p = x + v * V;
    int l = l0 + ty;
    for (; l + (kAhead - 1) * s.ty < l1; l += kAhead * s.ty) {
      typename Vec<T, V>::type e[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) e[j] = raw_v<T, V>(p + (int64_t)(l + j * s.ty) * a.xr);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) put(e[j], l + j * s.ty);
    }
    for (; l < l1; l += s.ty) put(raw_v<T, V>(p + (int64_t)l * a.xr), l);
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
  if (ty < s.ty) {
    for (int v = tx; v < s.cv; v += s.tx) {
      Affine<W, V> f;
      f.load(a.gamma, a.beta, v * V);
      float m[V], r[V], p[V], q[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int g = b * s.G + (v * V + i) / s.cpg;
        m[i] = a.mean[g];
        r[i] = a.rstd[g];
        p[i] = q[i] = 0.0f;
      }
      auto add = [&](const typename Vec<T, V>::type& xv, const typename Vec<T, V>::type& dv) {
        float e[V], d[V];
        widen<T, V>(xv, e);
        widen<T, V>(dv, d);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float xh;
          const float dz = grad_z<SILU>(e[i], d[i], m[i], r[i], f.ga[i], f.be[i], xh);
          p[i] += dz;
          q[i] = __builtin_fmaf(dz, xh, q[i]);
        }
      };
      const T* px = x + v * V;
      const T* pd = dy + v * V;
      int l = l0 + ty;
      for (; l + (kAhead - 1) * s.ty < l1; l += kAhead * s.ty) {
        typename Vec<T, V>::type e[kAhead], d[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          e[j] = raw_v<T, V>(px + (int64_t)(l + j * s.ty) * a.xr);
          d[j] = raw_v<T, V>(pd + (int64_t)(l + j * s.ty) * a.dyr);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) add(e[j], d[j]);
      }
      for (; l < l1; l += s.ty)
        add(raw_v<T, V>(px + (int64_t)l * a.xr), raw_v<T, V>(pd + (int64_t)l * a.dyr));
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

// dgamma and dbeta of channel c: sums over the images.
template <typename W>
__device__ __forceinline__ void sum_images(const float2* pq, int B, int C, int c, void* dgamma,
                                           void* dbeta) {
  if (c >= C) return;
  double p = 0.0, q = 0.0;
  for (int b = 0; b < B; ++b) {
    const float2 v = pq[(int64_t)b * C + c];
    p += v.x;
    q += v.y;
  }
  if (dgamma) reinterpret_cast<W*>(dgamma)[c] = (W)(float)q;
  if (dbeta) reinterpret_cast<W*>(dbeta)[c] = (W)(float)p;
}
template <typename W>
__global__ __launch_bounds__(256) void k_norm_sum_images(const float2* pq, int B, int C, void* dgamma,
                                                         void* dbeta) {
  sum_images<W>(pq, B, C, blockIdx.x * 256 + threadIdx.x, dgamma, dbeta);
}

template <typename T, typename W, int V, bool SILU>
__global__ __launch_bounds__(kNormThreads) void k_norm_grad_apply(GradK a) {
  const Shape& s = a.s;
  if ((int)blockIdx.x >= s.chunks) {
    if (blockIdx.y == 0)
      sum_images<W>(a.pq, s.B, s.C, ((int)blockIdx.x - s.chunks) * kNormThreads + threadIdx.x,
                    a.dgamma, a.dbeta);
    return;
  }
  const int tx = threadIdx.x % s.tx, ty = threadIdx.x / s.tx;
  if (ty >= s.ty) return;
  const int b = blockIdx.y, chunk = blockIdx.x;
  const int l0 = chunk * s.rows, l1 = min(s.L, l0 + s.rows);
  const T* x = reinterpret_cast<const T*>(a.x) + b * a.xb;
  const T* dy = reinterpret_cast<const T*>(a.dy) + b * a.dyb;
  T* dx = reinterpret_cast<T*>(a.dx) + b * a.dxb;
  for (int v = tx; v < s.cv; v += s.tx) {
    Affine<W, V> f;
    f.load(a.gamma, a.beta, v * V);
    float m[V], r[V], s1[V], s2[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int g = b * s.G + (v * V + i) / s.cpg;
      m[i] = a.mean[g];
      r[i] = a.rstd[g];
      const float2 t = a.s12[g];
      s1[i] = t.x;
      s2[i] = t.y;
    }
    auto put = [&](const typename Vec<T, V>::type& xv, const typename Vec<T, V>::type& dv, int l) {
      float e[V], d[V];
      widen<T, V>(xv, e);
      widen<T, V>(dv, d);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float xh;
        const float dz = grad_z<SILU>(e[i], d[i], m[i], r[i], f.ga[i], f.be[i], xh);
        e[i] = r[i] * (dz * f.ga[i] - s1[i] - xh * s2[i]);
      }
      store_v<T, V>(dx + (int64_t)l * a.dxr + v * V, e);
    };
    const T* px = x + v * V;
    const T* pd = dy + v * V;
    int l = l0 + ty;
    for (; l + (kAhead - 1) * s.ty < l1; l += kAhead * s.ty) {
      typename Vec<T, V>::type e[kAhead], d[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        e[j] = raw_v<T, V>(px + (int64_t)(l + j * s.ty) * a.xr);
        d[j] = raw_v<T, V>(pd + (int64_t)(l + j * s.ty) * a.dyr);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) put(e[j], d[j], l + j * s.ty);
    }
    for (; l < l1; l += s.ty)
      put(raw_v<T, V>(px + (int64_t)l * a.xr), raw_v<T, V>(pd + (int64_t)l * a.dyr), l);
  }
}

// ------------------------------------------------------------------- slabs ----
// One workgroup: one group of one image, [L, cpg] values at a row stride, in NV
// vectors a thread. Thread (tx, ty) has channel vector tx of positions ty,
// ty + TY, ...
struct SlabK {
  const void* x;
  int64_t xb, xr;
  const void* dy;
  int64_t dyb, dyr;
  void* y;  // y, or dx
  int64_t yb, yr;
  const void* gamma;
  const void* beta;
  float* mean;
  float* rstd;
  float2* pq;     // gradient: [B][C] sums of dz and dz xhat; nullptr with one image
  void* dgamma;   // gradient with one image
  void* dbeta;
  int B, L, C, G, cpg, vpr, ty;
  float eps;
};

// Workgroup to (image, group): neighbouring groups share cache lines, so one
// chiplet (ids go round the eight) gets neighbours.
__device__ __forceinline__ void slab_of(const SlabK& a, int id, int& b, int& g) {
  b = id / a.G;
  const int i = id % a.G;
  g = a.G % 8 == 0 ? (i % 8) * (a.G / 8) + i / 8 : i;
}

__device__ __forceinline__ float wave_sum(float v) {
  v += xor_lane<1>(v);
  v += xor_lane<2>(v);
  v += xor_lane<4>(v);
  v += xor_lane<8>(v);
  v += xor_lane<16>(v);
  return v + __shfl_xor(v, 32);
}

// Sums of two values over the workgroup, the waves' in fp64; valid in all threads.
__device__ __forceinline__ double2 slab_sum2(float u, float v, float2* lds) {
  u = wave_sum(u);
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = float2{u, v};
  __syncthreads();
  double2 s{0.0, 0.0};
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) {
    s.x += lds[w].x;
    s.y += lds[w].y;
  }
  return s;
}

template <typename T, typename W, int V, int NV, bool SILU>
__global__ __launch_bounds__(kNormThreads) void k_norm_slab(SlabK a) {
  __shared__ float2 red[kNormThreads / 64];
  int b, g;
  slab_of(a, blockIdx.x, b, g);
  const int tx = threadIdx.x % a.vpr, ty = threadIdx.x / a.vpr, c = g * a.cpg + tx * V;
  const bool live = ty < a.ty;
  const T* x = reinterpret_cast<const T*>(a.x) + b * a.xb + c;
  typename Vec<T, V>::type xv[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) xv[k] = raw_v<T, V>(x + (int64_t)min(ty + k * a.ty, a.L - 1) * a.xr);
  const float first = (float)(reinterpret_cast<const T*>(a.x) + b * a.xb)[g * a.cpg];
  Affine<W, V> f;
  f.load(a.gamma, a.beta, c);
  const double n = (double)a.L * a.cpg;
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (live && ty + k * a.ty < a.L) {
      float e[V];
      widen<T, V>(xv[k], e);
#pragma unroll
      for (int i = 0; i < V; ++i) s += e[i] - first;
    }
  const double md = (double)first + slab_sum2(s, 0.0f, red).x / n;
  const float m = (float)md;
  float q = 0.0f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (live && ty + k * a.ty < a.L) {
      float e[V];
      widen<T, V>(xv[k], e);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = e[i] - m;
        q = __builtin_fmaf(d, d, q);
      }
    }
  const double off = md - (double)m;  // squares about m, not about md
  const double var = variance(slab_sum2(q, 0.0f, red).x / n - off * off);
  const float r = (float)(1.0 / sqrt(var + (double)a.eps));
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[b * a.G + g] = m;
    if (a.rstd) a.rstd[b * a.G + g] = r;
  }
  T* y = reinterpret_cast<T*>(a.y) + b * a.yb + c;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int l = ty + k * a.ty;
    if (!live || l >= a.L) continue;
    float e[V];
    widen<T, V>(xv[k], e);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = act<SILU>(__builtin_fmaf(e[i] - m, r * f.ga[i], f.be[i]));
    store_v<T, V>(y + (int64_t)l * a.yr, e);
  }
}

template <typename T, typename W, int V, int NV, bool SILU>
__global__ __launch_bounds__(kNormThreads) void k_norm_slab_grad(SlabK a) {
  // With few workgroups arithmetic is what bounds this (a SiLU's gradient for every
  // value, twice): fp32 registers take xhat and dz gamma in place of x and dy.
  constexpr bool kKeep = sizeof(T) == 4;
  __shared__ float2 red[kNormThreads / 64];
  __shared__ float2 sums[kNormThreads * V];  // [ty][channel of the group]
  int b, g;
  slab_of(a, blockIdx.x, b, g);
  const int tx = threadIdx.x % a.vpr, ty = threadIdx.x / a.vpr, c = g * a.cpg + tx * V;
  const bool live = ty < a.ty;
  const T* x = reinterpret_cast<const T*>(a.x) + b * a.xb + c;
  const T* dy = reinterpret_cast<const T*>(a.dy) + b * a.dyb + c;
  typename Vec<T, V>::type xv[NV], dv[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int64_t l = min(ty + k * a.ty, a.L - 1);
    xv[k] = raw_v<T, V>(x + l * a.xr);
    dv[k] = raw_v<T, V>(dy + l * a.dyr);
  }
  Affine<W, V> f;
  f.load(a.gamma, a.beta, c);
  const float m = a.mean[b * a.G + g], r = a.rstd[b * a.G + g];
  float p[V], q[V];
#pragma unroll
  for (int i = 0; i < V; ++i) p[i] = q[i] = 0.0f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (live && ty + k * a.ty < a.L) {
      float e[V], d[V];
      widen<T, V>(xv[k], e);
      widen<T, V>(dv[k], d);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float xh;
        const float dz = grad_z<SILU>(e[i], d[i], m, r, f.ga[i], f.be[i], xh);
        p[i] += dz;
        q[i] = __builtin_fmaf(dz, xh, q[i]);
        if constexpr (kKeep) put_v<T, V>(xv[k], i, xh), put_v<T, V>(dv[k], i, dz * f.ga[i]);
      }
    }
  float u1 = 0.0f, u2 = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (live) sums[ty * a.cpg + tx * V + i] = float2{p[i], q[i]};
    u1 = __builtin_fmaf(f.ga[i], p[i], u1);
    u2 = __builtin_fmaf(f.ga[i], q[i], u2);
  }
  const double2 t = slab_sum2(u1, u2, red);  // its barriers publish `sums` too
  const double n = (double)a.L * a.cpg;
  const float s1 = (float)(t.x / n), s2 = (float)(t.y / n);
  // A channel's sums in two rounds where there are threads for it: `parts` threads
  // a channel, then one.
  const int parts = max(1, min((int)blockDim.x / a.cpg, 8));
  int rows = a.ty;
  if (parts > 1) {
    const int part = threadIdx.x / a.cpg, pc = threadIdx.x % a.cpg, len = (a.ty + parts - 1) / parts;
    float2 t{0.0f, 0.0f};
    if (part < parts)
      for (int y = part * len; y < min((part + 1) * len, a.ty); ++y) {
        t.x += sums[y * a.cpg + pc].x;
        t.y += sums[y * a.cpg + pc].y;
      }
    __syncthreads();
    if (part < parts) sums[part * a.cpg + pc] = t;
    __syncthreads();
    rows = parts;
  }
  for (int ch = threadIdx.x; ch < a.cpg; ch += blockDim.x) {
    float P = 0.0f, Q = 0.0f;
    for (int y = 0; y < rows; ++y) {
      P += sums[y * a.cpg + ch].x;
      Q += sums[y * a.cpg + ch].y;
    }
    if (a.pq) {
      a.pq[(int64_t)b * a.C + g * a.cpg + ch] = float2{P, Q};
    } else {
      if (a.dgamma) reinterpret_cast<W*>(a.dgamma)[g * a.cpg + ch] = (W)Q;
      if (a.dbeta) reinterpret_cast<W*>(a.dbeta)[g * a.cpg + ch] = (W)P;
    }
  }
  T* dx = reinterpret_cast<T*>(a.y) + b * a.yb + c;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int l = ty + k * a.ty;
    if (!live || l >= a.L) continue;
    float e[V], d[V];
    widen<T, V>(xv[k], e);
    widen<T, V>(dv[k], d);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float xh = e[i], t = d[i];
      if constexpr (!kKeep) t = grad_z<SILU>(e[i], d[i], m, r, f.ga[i], f.be[i], xh) * f.ga[i];
      e[i] = r * (t - s1 - xh * s2);
    }
    store_v<T, V>(dx + (int64_t)l * a.yr, e);
  }
}

bool rows_aligned(const void* p, int64_t sb, int64_t sr, int es, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (sb * es) % bytes == 0 &&
         (sr * es) % bytes == 0;
}

// Chunks for `groups` workgroups in all.
Shape shape_of(int B, int L, int C, int G, int V, int groups) {
  Shape s;
  s.B = B;
  s.L = L;
  s.C = C;
  s.G = G;
  s.cpg = C / G;
  s.cv = C / V;
  s.tx = s.cv < kNormThreads ? s.cv : kNormThreads;
  s.ty = kNormThreads / s.tx;
  const int step = kAhead * s.ty;
  int64_t want = (groups + B - 1) / B;
  const int64_t cap = ((int64_t)L + step - 1) / step;
  want = want < cap ? want : cap;
  s.rows = (int)(((int64_t)L + want - 1) / want);
  s.rows = (s.rows + step - 1) / step * step;
  s.chunks = (L + s.rows - 1) / s.rows;
  return s;
}
// Workgroups of the summing and of the writing launch. Measured (on one input again and
// again, which leaves more of it in the last-level cache) on 8x16384x320 bf16
// and on the gradient of 4x16383x256 bf16: summing with 256 / 512 / 1024: 61.6 / 61.8
// / 63.2 and 48.1 / 49.9 / 56.3 us; writing with 1024 / 2048 / 4096: 60.6 / 61.8 / 75.8
// and 50.1 / 49.9 / 49.9 us. Two and eight positions ahead instead of four: 67.2, 73.3
// and 55.4, 71.6 us.
constexpr int kSumGroups = 256, kApplyGroups = 1024;

template <typename T, typename W, int V>
hipError_t norm_run(const NormArgs& a, hipStream_t st) {
  const Shape s = shape_of(a.B, a.L, a.C, a.G, V, kSumGroups);
  double2* part = reinterpret_cast<double2*>(a.ws);
  float2* stats = reinterpret_cast<float2*>(part + (int64_t)s.B * s.chunks * s.G);
  const int threads = (s.tx * s.ty + 63) / 64 * 64;
  hipLaunchKernelGGL((k_norm_stats<T, V>), dim3(s.chunks, s.B), dim3(threads),
                     (size_t)s.ty * s.C * sizeof(float2), st, StatsK{a.x, a.xb, a.xr, part, s});
  hipLaunchKernelGGL(k_norm_stats_join, dim3((s.B * s.G + 3) / 4), dim3(256), 0, st, part,
                     StatsOut{stats, a.mean, a.rstd, a.eps}, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const Shape t = shape_of(a.B, a.L, a.C, a.G, V, kApplyGroups);
  const ApplyK k{a.x, a.xb, a.xr, a.y, a.yb, a.yr, a.gamma, a.beta, stats, t};
  if (a.act)
    hipLaunchKernelGGL((k_norm_apply<T, W, V, true>), dim3(t.chunks, t.B), dim3(threads), 0, st, k);
  else
    hipLaunchKernelGGL((k_norm_apply<T, W, V, false>), dim3(t.chunks, t.B), dim3(threads), 0, st, k);
  return hipGetLastError();
}

template <typename T, typename W, int V>
hipError_t norm_grad_run(const NormArgs& a, hipStream_t st) {
  const bool empty = a.B == 0 || a.L == 0;  // dgamma and dbeta are still written: zero
  float2* pq = reinterpret_cast<float2*>(a.ws);
  if (empty) {
    hipLaunchKernelGGL(k_norm_sum_images<W>, dim3((a.C + 255) / 256), dim3(256), 0, st, pq, 0, a.C,
                       a.dgamma, a.dbeta);
    return hipGetLastError();
  }
  const Shape s = shape_of(a.B, a.L, a.C, a.G, V, kSumGroups);
  float2* s12 = pq + (int64_t)s.B * s.C;
  float2* part = s12 + (int64_t)s.B * s.G;
  GradK k{a.x,    a.xb,   a.xr, a.dy, a.dyb, a.dyr,    a.y,     a.yb, a.yr, a.gamma, a.beta,
          a.mean, a.rstd, part, pq,   s12,   a.dgamma, a.dbeta, s};
  const int threads = (s.tx * s.ty + 63) / 64 * 64;
  const size_t lds = (size_t)s.ty * s.C * sizeof(float2);
  if (a.act)
    hipLaunchKernelGGL((k_norm_grad_sums<T, W, V, true>), dim3(s.chunks, s.B), dim3(threads), lds,
                       st, k);
  else
    hipLaunchKernelGGL((k_norm_grad_sums<T, W, V, false>), dim3(s.chunks, s.B), dim3(threads), lds,
                       st, k);
  hipLaunchKernelGGL(k_norm_grad_reduce<W>, dim3(s.B * s.G), dim3(256), 0, st, k);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k.s = shape_of(a.B, a.L, a.C, a.G, V, kApplyGroups);
  const dim3 grid(k.s.chunks + (s.C + kNormThreads - 1) / kNormThreads, s.B);
  if (a.act)
    hipLaunchKernelGGL((k_norm_grad_apply<T, W, V, true>), grid, dim3(kNormThreads), 0, st, k);
  else
    hipLaunchKernelGGL((k_norm_grad_apply<T, W, V, false>), grid, dim3(kNormThreads), 0, st, k);
  return hipGetLastError();
}

// Tensors that go by slabs with vectors narrower than 16 bytes too.
bool small_tensor(int B, int L, int C, int es) { return (int64_t)B * L * C * es <= 24 << 20; }

// Vectors a thread holds when one workgroup takes a slab, 0 where it does not fit.
template <typename T, int V>
int slab_vectors(const NormArgs& a) {
  const int cpg = a.C / a.G;
  if (cpg % V != 0 || cpg / V > kNormThreads || a.B == 0 || a.L == 0) return 0;
  const int ty = kNormThreads / (cpg / V);
  const int64_t nv = ((int64_t)a.L + ty - 1) / ty;
  return nv <= slab_most(V * (int)sizeof(T)) ? (int)nv : 0;
}

template <typename T, typename W, int V, int NV>
hipError_t slab_run(const NormArgs& a, bool grad, hipStream_t st) {
  SlabK k{};
  k.x = a.x;
  k.xb = a.xb;
  k.xr = a.xr;
  k.dy = a.dy;
  k.dyb = a.dyb;
  k.dyr = a.dyr;
  k.y = a.y;
  k.yb = a.yb;
  k.yr = a.yr;
  k.gamma = a.gamma;
  k.beta = a.beta;
  k.mean = a.mean;
  k.rstd = a.rstd;
  k.dgamma = a.dgamma;
  k.dbeta = a.dbeta;
  k.pq = grad && a.B > 1 ? reinterpret_cast<float2*>(a.ws) : nullptr;
  k.B = a.B;
  k.L = a.L;
  k.C = a.C;
  k.G = a.G;
  k.cpg = a.C / a.G;
  k.vpr = k.cpg / V;
  k.eps = a.eps;
  // no more threads than positions ask for
  const int most = kNormThreads / k.vpr;
  const int need = (a.L + NV - 1) / NV;
  k.ty = most < need ? most : need;
  const dim3 grid(a.B * a.G), block((k.vpr * k.ty + 63) / 64 * 64);
  if (!grad) {
    if (a.act)
      hipLaunchKernelGGL((k_norm_slab<T, W, V, NV, true>), grid, block, 0, st, k);
    else
      hipLaunchKernelGGL((k_norm_slab<T, W, V, NV, false>), grid, block, 0, st, k);
    return hipGetLastError();
  }
  if (a.act)
    hipLaunchKernelGGL((k_norm_slab_grad<T, W, V, NV, true>), grid, block, 0, st, k);
  else
    hipLaunchKernelGGL((k_norm_slab_grad<T, W, V, NV, false>), grid, block, 0, st, k);
  if (k.pq && (a.dgamma || a.dbeta))
    hipLaunchKernelGGL(k_norm_sum_images<W>, dim3((a.C + 255) / 256), dim3(256), 0, st, k.pq, a.B,
                       a.C, a.dgamma, a.dbeta);
  return hipGetLastError();
}

template <typename T, typename W, int V>
hipError_t norm_width(const NormArgs& a, bool slabs, bool grad, hipStream_t st) {
  const int nv = slabs ? slab_vectors<T, V>(a) : 0;
  if (nv > 0) {
    constexpr int most = slab_most(V * (int)sizeof(T));
    if (nv <= 3) return slab_run<T, W, V, 3>(a, grad, st);
    if (nv <= 6) return slab_run<T, W, V, 6>(a, grad, st);
    if (nv <= 12) return slab_run<T, W, V, 12>(a, grad, st);
    if constexpr (most >= 24) {
      if (nv <= 24) return slab_run<T, W, V, 24>(a, grad, st);
    }
    if constexpr (most >= 48) return slab_run<T, W, V, 48>(a, grad, st);
  }
  return grad ? norm_grad_run<T, W, V>(a, st) : norm_run<T, W, V>(a, st);
}

template <typename T, typename W>
hipError_t norm_dispatch(const NormArgs& a, bool grad, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const int es = sizeof(T), cpg = a.C / a.G;
  auto aligned = [&](int bytes) {
    return a.C * es % bytes == 0 && rows_aligned(a.x, a.xb, a.xr, es, bytes) &&
           rows_aligned(a.y, a.yb, a.yr, es, bytes) &&
           (!grad || rows_aligned(a.dy, a.dyb, a.dyr, es, bytes));
  };
  // A slab's rows have cpg channels: the widest vector that divides them. Narrow
  // vectors cost the load path more, so with them only tensors of up to 24 MiB go
  // by slabs. Measured, slabs / two readings: 8x2048x640 bf16 (8-byte vectors, 21 MB)
  // 18.0 / 29.4 us; 16x1024x320 bf16 (4 bytes, 10 MB) 13.8 / 23.9; 16x4096x320 bf16
  // (4 bytes, 42 MB) 50.8 / 37.5; 2x500x224 bf16 (2 bytes, 0.4 MB) 12.9 / 17.9;
  // gradients of 2x500x224 bf16 15.3 / 23.7 and of 16x2048x320 fp32 (8 bytes, 42 MB)
  // 52.1 / 44.3.
  const bool small = small_tensor(a.B, a.L, a.C, es);
  if (aligned(16) && slab_vectors<T, V>(a)) return norm_width<T, W, V>(a, true, grad, st);
  if (small && aligned(8) && cpg % (V / 2) == 0 && slab_vectors<T, V / 2>(a))
    return norm_width<T, W, V / 2>(a, true, grad, st);
  if (small && V == 8 && aligned(4) && slab_vectors<T, 2>(a))
    return norm_width<T, W, 2>(a, true, grad, st);
  if (small && slab_vectors<T, 1>(a)) return norm_width<T, W, 1>(a, true, grad, st);
  if (aligned(16)) return norm_width<T, W, V>(a, false, grad, st);
  return norm_width<T, W, 1>(a, false, grad, st);
}

hipError_t norm_types(const NormArgs& a, bool grad, hipStream_t s) {
  if (a.x_bf16)
    return a.w_bf16 ? norm_dispatch<bf16, bf16>(a, grad, s) : norm_dispatch<bf16, float>(a, grad, s);
  return a.w_bf16 ? norm_dispatch<float, bf16>(a, grad, s) : norm_dispatch<float, float>(a, grad, s);
}

}  // namespace

int64_t norm_ws_bytes(int B, int L, int C, int G, int es, bool grad) {
  // Small tensors whose slabs fit even element by element go by slabs at any
  // alignment: the gradient's per-channel sums are all they put through memory.
  const int cpg = C / G;
  if (small_tensor(B, L, C, es) && cpg <= kNormThreads &&
      ((int64_t)L + kNormThreads / cpg - 1) / (kNormThreads / cpg) <= slab_most(es))
    return grad && B > 1 ? (int64_t)B * C * (int64_t)sizeof(float2) : 0;
  int64_t chunks = 0;  // the most of any vector width
  for (int V : {1, 2, 4, 8}) {
    if (C % V) continue;
    const Shape s = shape_of(B, L, C, G, V, kSumGroups);
    chunks = chunks > s.chunks ? chunks : s.chunks;
  }
  if (!grad)
    return (int64_t)B * G * (chunks * (int64_t)sizeof(double2) + (int64_t)sizeof(float2));
  return ((int64_t)B * C + (int64_t)B * G + (int64_t)B * chunks * C) * (int64_t)sizeof(float2);
}

hipError_t launch_group_norm(const NormArgs& a, hipStream_t s) {
  if (a.L > 0) return norm_types(a, false, s);
  Shape e{};  // no positions: 0 / 0 for the statistics, no outputs
  e.B = a.B;
  e.G = a.G;
  e.cpg = a.C / a.G;
  hipLaunchKernelGGL(k_norm_stats_join, dim3((a.B * a.G + 3) / 4), dim3(256), 0, s, nullptr,
                     StatsOut{nullptr, a.mean, a.rstd, a.eps}, e);
  return hipGetLastError();
}

hipError_t launch_group_norm_grad(const NormArgs& a, hipStream_t s) {
  return norm_types(a, true, s);
}

}  // namespace ql
