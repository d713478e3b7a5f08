// Norms of queries and keys for each head and their rotation by positions of
// several axes, in one pass behind the qkv linear, forward and backward.
//
//   forward   n = x rstd gamma, rstd = 1 / sqrt(mean x^2 + eps);  a pair (a, b) of n
//             becomes (a cos - b sin, a sin + b cos) of position times frequency
//   backward  dn = the pairs of dy turned back;  dgamma = sum dn x rstd;
//             dx = rstd (dn gamma - x rstd^2 mean(dn gamma x))
//
// Bound by memory: some 10 operations an element that is read and written. G lanes
// share a head, lane j taking the 16-byte pieces j, j + G, ... of it, so that neighbouring
// lanes read neighbouring addresses and a head's sums cross two or three lanes. The
// angles are the same for all heads of a token: a workgroup forms the sines and
// cosines of its tokens once, in LDS, a pair a thread (fp64 up to the fraction of a turn).
#include "ql_block.h"
#include "ql_device.h"

namespace ql {

namespace {

typedef __bf16 bf16;
constexpr int kThreads = 256;
constexpr int kMaxTokens = 64;
constexpr int kMaxPairs = 80;

template <typename T, int N>
struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Vec {
  T e[N];
};

__device__ __forceinline__ float read_w(const void* p, bool is_bf16, int i) {
  return is_bf16 ? (float)reinterpret_cast<const bf16*>(p)[i] : reinterpret_cast<const float*>(p)[i];
}

// Pairs are numbered axis by axis, then those that do not turn (numbered like one more
// axis). Channels of pair p, and its axis (n_axes: does not turn).
__device__ __forceinline__ int pair_channels(const HeadsArgs& a, int p, int& c1, int& c2) {
  int axis = 0, first = 0, half = a.D / 2;
#pragma unroll
  for (int i = 0; i < QL_MAX_AXES; ++i)
    if (i < a.n_axes && axis == i && p - first >= a.half[i]) {
      first += a.half[i];
      axis = i + 1;
    }
  half = axis < a.n_axes ? a.half[axis] : a.D / 2 - first;
  c1 = a.halves ? 2 * first + (p - first) : 2 * p;
  c2 = a.halves ? c1 + half : c1 + 1;
  return axis;
}

// How a lane's pairs lie: one vector of neighbouring pairs (a, b, a, b), one of first
// and one of second members, or anyhow.
enum { kAdjacent = 0, kHalves = 1, kScattered = 2 };

template <typename XT> struct Geo {
  static constexpr int V = 16 / sizeof(XT), P = V / 2;  // channels and pairs of a piece
};

// Where the pieces of a lane lie in a head, in pair order.
template <int C, int P, int MODE>
struct Places {
  int c1[MODE == kScattered ? C * P : C], c2[MODE == kScattered ? C * P : C];
  int pieces, j;
  template <int G>
  __device__ __forceinline__ void find(const HeadsArgs& a, int lane_in_head) {
    j = lane_in_head;
    pieces = a.D / (2 * P);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int u = min(j + c * G, pieces - 1);
      if constexpr (MODE == kScattered) {
#pragma unroll
        for (int i = 0; i < P; ++i) pair_channels(a, u * P + i, c1[c * P + i], c2[c * P + i]);
      } else {
        pair_channels(a, u * P, c1[c], c2[c]);
      }
    }
  }
};

// Values of a lane: pairs (p[.][.][0], p[.][.][1]); pieces past the head are zero.
template <int C, int P>
struct Vals {
  float p[C][P][2];
};

template <typename T, int C, int P, int G, int MODE>
__device__ __forceinline__ void load(const T* row, const Places<C, P, MODE>& w, bool ok,
                                     Vals<C, P>& v) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const bool in = ok && w.j + c * G < w.pieces;
#pragma unroll
    for (int i = 0; i < P; ++i) v.p[c][i][0] = v.p[c][i][1] = 0.0f;
    if (!in) continue;
    if constexpr (MODE == kAdjacent) {
      const Vec<T, 2 * P> x = *reinterpret_cast<const Vec<T, 2 * P>*>(row + w.c1[c]);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        v.p[c][i][0] = (float)x.e[2 * i];
        v.p[c][i][1] = (float)x.e[2 * i + 1];
      }
    } else if constexpr (MODE == kHalves) {
      const Vec<T, P> x = *reinterpret_cast<const Vec<T, P>*>(row + w.c1[c]);
      const Vec<T, P> y = *reinterpret_cast<const Vec<T, P>*>(row + w.c2[c]);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        v.p[c][i][0] = (float)x.e[i];
        v.p[c][i][1] = (float)y.e[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        v.p[c][i][0] = (float)row[w.c1[c * P + i]];
        v.p[c][i][1] = (float)row[w.c2[c * P + i]];
      }
    }
  }
}

template <typename T, int C, int P, int G, int MODE>
__device__ __forceinline__ void store(T* row, const Places<C, P, MODE>& w, const Vals<C, P>& v) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (w.j + c * G >= w.pieces) continue;
    if constexpr (MODE == kAdjacent) {
      Vec<T, 2 * P> x;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        x.e[2 * i] = (T)v.p[c][i][0];
        x.e[2 * i + 1] = (T)v.p[c][i][1];
      }
      *reinterpret_cast<Vec<T, 2 * P>*>(row + w.c1[c]) = x;
    } else if constexpr (MODE == kHalves) {
      Vec<T, P> x, y;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        x.e[i] = (T)v.p[c][i][0];
        y.e[i] = (T)v.p[c][i][1];
      }
      *reinterpret_cast<Vec<T, P>*>(row + w.c1[c]) = x;
      *reinterpret_cast<Vec<T, P>*>(row + w.c2[c]) = y;
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        row[w.c1[c * P + i]] = (T)v.p[c][i][0];
        row[w.c2[c * P + i]] = (T)v.p[c][i][1];
      }
    }
  }
}

template <int G>
__device__ __forceinline__ float head_sum(float v) {
  v += xor_lane<1>(v);
  v += xor_lane<2>(v);
  if constexpr (G >= 8) v += xor_lane<4>(v);
  if constexpr (G >= 16) v += xor_lane<8>(v);
  return v;
}

// Cosines and sines of `n` tokens from `tok0` on into turn[token][pair].
__device__ __forceinline__ void form_turns(const HeadsArgs& a, float2* turn, int64_t tok0, int n) {
  const int pairs = a.D / 2;
  for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
    const int t = i / pairs, p = i - t * pairs;
    int c1, c2;
    const int axis = pair_channels(a, p, c1, c2);
    float2 cs = make_float2(1.0f, 0.0f);
    if (axis < a.n_axes) {
      const int tok = (int)tok0 + t, b = tok / a.L;
      const int64_t at = b * a.pb + (int64_t)(tok - b * a.L) * a.n_axes + axis;
      const double x = a.pos_f32 ? (double)reinterpret_cast<const float*>(a.pos)[at]
                                 : (double)reinterpret_cast<const int32_t*>(a.pos)[at];
      const double turns = x * a.freqs[p];
      const float part = (float)(turns - rint(turns));
      sincospif(2.0f * part, &cs.y, &cs.x);
    }
    turn[i] = cs;
  }
}

// Where the tokens' rows start, in elements: x and dx, and the outputs or their gradients.
struct Starts {
  int64_t x, dx, y[3];
};
__device__ __forceinline__ void find_starts(const HeadsArgs& a, Starts* out, int64_t tok0, int n) {
  for (int t = threadIdx.x; t < n; t += kThreads) {
    const int tok = (int)tok0 + t, b = tok / a.L, l = tok - b * a.L;
    Starts s;
    s.x = b * a.xb + l * a.xr;
    s.dx = b * a.db + l * a.dr;
#pragma unroll
    for (int i = 0; i < 3; ++i) s.y[i] = b * a.y[i].batch + l * a.y[i].row;
    out[t] = s;
  }
}

// The gammas in pair order: out[part][2 pair + member].
__device__ __forceinline__ void fetch_gammas(const HeadsArgs& a, float (*out)[2 * kMaxPairs]) {
  for (int i = threadIdx.x; i < a.D; i += kThreads) {
    const int part = i / (a.D / 2), p = i - part * (a.D / 2);
    int c1, c2;
    pair_channels(a, p, c1, c2);
    const void* g = a.gamma[part];
    out[part][2 * p] = g ? read_w(g, a.w_bf16, c1) : 1.0f;
    out[part][2 * p + 1] = g ? read_w(g, a.w_bf16, c2) : 1.0f;
  }
}

// ----------------------------------------------------------------- forward ----

template <typename XT, typename YT, int G, int C, int MODE>
__global__ __launch_bounds__(kThreads) void k_heads(HeadsArgs a) {
  constexpr int P = Geo<XT>::P, kGroups = kThreads / G;
  __shared__ float gamma[2][2 * kMaxPairs];
  __shared__ Starts starts[kMaxTokens];
  extern __shared__ float2 turn[];  // [tokens][D / 2]
  const int tid = threadIdx.x, group = tid / G;
  const int64_t all = (int64_t)a.B * a.L, tok0 = (int64_t)blockIdx.x * a.tokens;
  const int n = (int)(all - tok0 < a.tokens ? all - tok0 : a.tokens);
  const int heads = a.heads[0] + a.heads[1] + a.heads[2], rows = n * heads;
  find_starts(a, starts, tok0, n);
  Places<C, P, MODE> at;
  at.template find<G>(a, tid % G);
  __syncthreads();
  const auto row_in = [&](int r) {
    const int t = r / heads;
    return reinterpret_cast<const XT*>(a.x) + starts[t].x + (r - t * heads) * a.D;
  };
  Vals<C, P> v, next;
  load<XT, C, P, G, MODE>(row_in(min(group, rows - 1)), at, group < rows, next);
  fetch_gammas(a, gamma);
  form_turns(a, turn, tok0, n);
  __syncthreads();
  for (int r = group; r < rows; r += kGroups) {
    v = next;
    const int rn = r + kGroups;
    load<XT, C, P, G, MODE>(row_in(min(rn, rows - 1)), at, rn < rows, next);
    const int t = r / heads;
    int hd = r - t * heads;
    const int part = hd < a.heads[0] ? 0 : hd < a.heads[0] + a.heads[1] ? 1 : 2;
    if (part == 1) hd -= a.heads[0];
    if (part == 2) hd -= a.heads[0] + a.heads[1];
    if (part < 2) {
      float rstd = 1.0f;
      if (a.rms) {
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < P; ++i)
            sum = __builtin_fmaf(v.p[c][i][0], v.p[c][i][0],
                                 __builtin_fmaf(v.p[c][i][1], v.p[c][i][1], sum));
        rstd = rsqrtf(head_sum<G>(sum) / (float)a.D + a.eps);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int p0 = min(at.j + c * G, at.pieces - 1) * P;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float2 cs = turn[t * (a.D / 2) + p0 + i];
          float x = v.p[c][i][0], y = v.p[c][i][1];
          if (a.rms) {
            x *= rstd * gamma[part][2 * (p0 + i)];
            y *= rstd * gamma[part][2 * (p0 + i) + 1];
          }
          v.p[c][i][0] = __builtin_fmaf(x, cs.x, -(y * cs.y));
          v.p[c][i][1] = __builtin_fmaf(x, cs.y, y * cs.x);
        }
      }
    }
    store<YT, C, P, G, MODE>(reinterpret_cast<YT*>(a.y[part].p) + starts[t].y[part] +
                                 hd * a.y[part].head,
                             at, v);
  }
}

// ---------------------------------------------------------------- backward ----

// blockIdx.y says which part (q, k, v) a workgroup works for, so that a lane keeps
// one sum of dgamma; it walks over the tokens in steps of gridDim.x tiles.
template <typename XT, typename YT, int G, int C, int MODE>
__global__ __launch_bounds__(kThreads) void k_heads_grad(HeadsArgs a) {
  constexpr int P = Geo<XT>::P, kGroups = kThreads / G;
  __shared__ float gamma[2][2 * kMaxPairs];
  __shared__ float sums[kThreads / 64][2 * kMaxPairs];
  __shared__ Starts starts[kMaxTokens];
  extern __shared__ float2 turn[];
  const int tid = threadIdx.x, group = tid / G, part = blockIdx.y, heads = a.heads[part];
  const int64_t all = (int64_t)a.B * a.L;
  const int head0 = part == 0 ? 0 : part == 1 ? a.heads[0] : a.heads[0] + a.heads[1];
  Places<C, P, MODE> at;
  at.template find<G>(a, tid % G);
  fetch_gammas(a, gamma);
  Vals<C, P> dg;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < P; ++i) dg.p[c][i][0] = dg.p[c][i][1] = 0.0f;
  const ql_heads_view& y = a.y[part];
  const int64_t step = (int64_t)gridDim.x * a.tokens;
  for (int64_t tok0 = (int64_t)blockIdx.x * a.tokens; tok0 < all && heads > 0; tok0 += step) {
    const int n = (int)(all - tok0 < a.tokens ? all - tok0 : a.tokens), rows = n * heads;
    __syncthreads();  // the turns before have been read
    find_starts(a, starts, tok0, n);
    if (part < 2) form_turns(a, turn, tok0, n);
    __syncthreads();
    for (int r = group; r < rows; r += kGroups) {
      const int t = r / heads, hd = r - t * heads;
      Vals<C, P> x, d;
      load<YT, C, P, G, MODE>(reinterpret_cast<const YT*>(y.p) + starts[t].y[part] + hd * y.head, at,
                              true, d);
      if (part < 2) {
        if (a.rms)
          load<XT, C, P, G, MODE>(reinterpret_cast<const XT*>(a.x) + starts[t].x +
                                      (head0 + hd) * a.D, at, true, x);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int p0 = min(at.j + c * G, at.pieces - 1) * P;
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const float2 cs = turn[t * (a.D / 2) + p0 + i];
            const float da = d.p[c][i][0], db = d.p[c][i][1];
            d.p[c][i][0] = __builtin_fmaf(da, cs.x, db * cs.y);
            d.p[c][i][1] = __builtin_fmaf(db, cs.x, -(da * cs.y));
          }
        }
        if (a.rms) {
          float s2 = 0.0f, st = 0.0f;
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const int p0 = min(at.j + c * G, at.pieces - 1) * P;
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float xv = x.p[c][i][e];
                s2 = __builtin_fmaf(xv, xv, s2);
                st = __builtin_fmaf(d.p[c][i][e] * gamma[part][2 * (p0 + i) + e], xv, st);
              }
          }
          s2 = head_sum<G>(s2);
          st = head_sum<G>(st);
          const float rstd = rsqrtf(s2 / (float)a.D + a.eps);
          const float f = rstd * rstd * (st / (float)a.D);
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const int p0 = min(at.j + c * G, at.pieces - 1) * P;
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float dn = d.p[c][i][e], xv = x.p[c][i][e];
                dg.p[c][i][e] = __builtin_fmaf(dn, xv * rstd, dg.p[c][i][e]);
                d.p[c][i][e] = rstd * __builtin_fmaf(dn, gamma[part][2 * (p0 + i) + e], -(xv * f));
              }
          }
        }
      }
      store<XT, C, P, G, MODE>(reinterpret_cast<XT*>(a.dx) + starts[t].dx + (head0 + hd) * a.D, at, d);
    }
  }
  if (!a.part || part == 2) return;
  // lanes of the same pieces, then waves
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = dg.p[c][i][e];
        if constexpr (G <= 4) v += __shfl_xor(v, 4);
        if constexpr (G <= 8) v += __shfl_xor(v, 8);
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
        if ((tid & 63) < G && at.j + c * G < at.pieces)
          sums[tid >> 6][2 * ((at.j + c * G) * P + i) + e] = v;
      }
  __syncthreads();
  for (int i = tid; i < a.D; i += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) v += sums[w][i];
    a.part[((int64_t)part * gridDim.x + blockIdx.x) * a.D + i] = v;  // in pair order
  }
}

// dgamma of part blockIdx.y, 32 channels a workgroup, from the workgroups' sums: 32 strips
// of them, eight loads in flight.
__global__ __launch_bounds__(1024) void k_heads_gamma(HeadsArgs a) {
  __shared__ double box[16][32];
  const int part = blockIdx.y, col = threadIdx.x % 32, i = blockIdx.x * 32 + col;
  const int strip = threadIdx.x / 32;
  if (!a.dgamma[part]) return;
  double sum = 0.0;
  if (i < a.D) {
    const float* p = a.part + (int64_t)part * a.groups * a.D + i;
    for (int g = strip; g < a.groups; g += 256) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = g + 32 * j < a.groups ? p[(int64_t)(g + 32 * j) * a.D] : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += (double)v[j];
    }
  }
  sum += __shfl_xor(sum, 32);  // two strips a wave
  if (strip % 2 == 0) box[strip / 2][col] = sum;
  __syncthreads();
  if (strip > 1) return;
  sum = 0.0;
#pragma unroll
  for (int s = 0; s < 8; ++s) sum += box[8 * strip + s][col];
  sum += __shfl_xor(sum, 32);
  if (strip != 0 || i >= a.D) return;
  int c1, c2;
  pair_channels(a, i / 2, c1, c2);
  const int c = i % 2 ? c2 : c1;
  if (a.w_bf16)
    reinterpret_cast<bf16*>(a.dgamma[part])[c] = (bf16)(float)sum;
  else
    reinterpret_cast<float*>(a.dgamma[part])[c] = (float)sum;
}

// ------------------------------------------------------------------ launch ----

template <typename XT>
int mode_of(const HeadsArgs& a) {
  if (!a.vec) return kScattered;
  if (!a.halves) return kAdjacent;
  int rest = a.D / 2;
  for (int i = 0; i < a.n_axes; ++i) {
    if (a.half[i] % Geo<XT>::P) return kScattered;
    rest -= a.half[i];
  }
  return rest % Geo<XT>::P ? kScattered : kHalves;
}

template <typename XT, typename YT, int G, int C>
hipError_t run(const HeadsArgs& a, bool grad, dim3 grid, hipStream_t s) {
  const size_t lds = (size_t)a.tokens * (a.D / 2) * sizeof(float2);
  const int mode = mode_of<XT>(a);
#define QL_HEADS_MODE(M)                                      \
  if (mode == M) {                                            \
    if (grad)                                                 \
      k_heads_grad<XT, YT, G, C, M><<<grid, kThreads, lds, s>>>(a); \
    else                                                      \
      k_heads<XT, YT, G, C, M><<<grid, kThreads, lds, s>>>(a);   \
  }
  QL_HEADS_MODE(kAdjacent)
  QL_HEADS_MODE(kHalves)
  QL_HEADS_MODE(kScattered)
#undef QL_HEADS_MODE
  return hipGetLastError();
}

// Lanes of a head: as few as keep a lane's values in registers with room for other waves,
// twice as many where the pieces still fill them.
template <typename XT>
int lanes_of(int D) { return (D % 64 == 0 ? 2 : 1) * (sizeof(XT) == 4 ? 8 : 4); }

template <typename XT, typename YT>
hipError_t pick(const HeadsArgs& a, bool grad, dim3 grid, hipStream_t s) {
  constexpr int G = sizeof(XT) == 4 ? 8 : 4;
  if (a.D == 64) return run<XT, YT, 2 * G, 1>(a, grad, grid, s);
  if (a.D == 128) return run<XT, YT, 2 * G, 2>(a, grad, grid, s);
  switch ((a.D + 31) / 32) {
    case 1: return run<XT, YT, G, 1>(a, grad, grid, s);
    case 2: return run<XT, YT, G, 2>(a, grad, grid, s);
    case 3: return run<XT, YT, G, 3>(a, grad, grid, s);
    case 4: return run<XT, YT, G, 4>(a, grad, grid, s);
    default: return run<XT, YT, G, 5>(a, grad, grid, s);
  }
}

hipError_t go(const HeadsArgs& a, bool grad, dim3 grid, hipStream_t s) {
  if (a.x_bf16)
    return a.y_bf16 ? pick<bf16, bf16>(a, grad, grid, s) : pick<bf16, float>(a, grad, grid, s);
  return a.y_bf16 ? pick<float, bf16>(a, grad, grid, s) : pick<float, float>(a, grad, grid, s);
}

// Tokens of a workgroup: enough rows for four passes of its lanes, unless that
// leaves fewer workgroups than fill the chip.
int tokens_of(int64_t all, int heads, int D, bool x_bf16) {
  const int groups = kThreads / (x_bf16 ? lanes_of<bf16>(D) : lanes_of<float>(D));
  int t = 1;
  while (t < kMaxTokens && t * heads < 4 * groups &&
         (t * heads < groups || all / (2 * t) >= 1024))
    t *= 2;
  return t;
}

}  // namespace

int heads_grad_groups(int64_t tokens, int heads) {
  (void)heads;
  return (int)(tokens < 512 ? (tokens < 1 ? 1 : tokens) : 512);
}

hipError_t launch_heads(const HeadsArgs& args, hipStream_t s) {
  HeadsArgs a = args;
  const int64_t all = (int64_t)a.B * a.L;
  a.tokens = tokens_of(all, a.heads[0] + a.heads[1] + a.heads[2], a.D, a.x_bf16);
  return go(a, false, dim3((unsigned)((all + a.tokens - 1) / a.tokens)), s);
}

hipError_t launch_heads_grad(const HeadsArgs& args, hipStream_t s) {
  HeadsArgs a = args;
  const int64_t all = (int64_t)a.B * a.L;
  if (all > 0) {
    const int most = a.heads[0] > a.heads[1] ? a.heads[0] : a.heads[1];
    a.tokens = tokens_of(all, most > a.heads[2] ? most : a.heads[2], a.D, a.x_bf16);
    const hipError_t e = go(a, true, dim3((unsigned)a.groups, 3), s);
    if (e != hipSuccess) return e;
  }
  if (!a.dgamma[0] && !a.dgamma[1]) return hipSuccess;
  if (all == 0) a.groups = 0;
  k_heads_gamma<<<dim3((a.D + 31) / 32, 2), 1024, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ql
