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
// lanes read neighbouring addresses and a head's sums cross two to four lanes. The
// angles are the same for all heads of a token: a workgroup forms the sines and
// cosines of its tokens once, in LDS (fp64 up to the fraction of a turn), signed so that
// every channel becomes n[c] cos + n[partner] sin. Adjacent partners are in the lane; any
// others trade places in LDS (read and written in halves of pieces, with the
// partners in one lane, the clip below takes 95 us where heads are cut at multiples of
// four pairs, and element by element, as other heads would need, 213).
//
// Measured: one clip, 17550 tokens of 32 + 4 + 4 heads of 128, bf16: 97-102 us, 3.5-3.7 TB/s, for
// pairs in halves (LDS is busy 64 % of it, 38 % with conflicts), 78 (4.6) for neighbours;
// gradient, 18432 tokens of 3 x 16 heads of 128, bf16: 132 us, 5.1 TB/s, and 7 for the sum of dgamma.
#include "ql_block.h"
#include "ql_device.h"

namespace ql {

namespace {

typedef __bf16 bf16;
constexpr int kThreads = 256;
constexpr int kMaxTokens = 32;  // their turns take up to 40 KB of LDS
constexpr int kMaxDim = 160;

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
  int axis = 0, first = 0;
#pragma unroll
  for (int i = 0; i < QL_MAX_AXES; ++i)
    if (i < a.n_axes && axis == i && p - first >= a.half[i]) {
      first += a.half[i];
      axis = i + 1;
    }
  const int half = axis < a.n_axes ? a.half[axis] : a.D / 2 - first;
  c1 = a.halves ? 2 * first + (p - first) : 2 * p;
  c2 = a.halves ? c1 + half : c1 + 1;
  return axis;
}

// How partners meet and rows are read: pairs of neighbours, in vectors; any pairs, in
// vectors; any pairs, element by element (rows that no vector is aligned to).
enum { kAdjacent = 0, kApart = 1, kByElement = 2 };

// Channels of a piece.
template <typename XT> constexpr int kV = 16 / sizeof(XT);

// Values of a lane: piece c has channels (j + c G) V .. + V - 1; those past the head are 0.
template <int C, int V>
struct Vals {
  float v[C][V];
};

template <typename T, int C, int V, int G, int MODE>
__device__ __forceinline__ void load(const T* row, int j, int pieces, bool ok, Vals<C, V>& x) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int u = j + c * G;
    if (ok && u < pieces) {
      if constexpr (MODE == kByElement) {
#pragma unroll
        for (int i = 0; i < V; ++i) x.v[c][i] = (float)row[u * V + i];
      } else {
        const Vec<T, V> y = *reinterpret_cast<const Vec<T, V>*>(row + u * V);
#pragma unroll
        for (int i = 0; i < V; ++i) x.v[c][i] = (float)y.e[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) x.v[c][i] = 0.0f;
    }
  }
}

template <typename T, int C, int V, int G, int MODE>
__device__ __forceinline__ void store(T* row, int j, int pieces, const Vals<C, V>& x) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int u = j + c * G;
    if (u >= pieces) continue;
    if constexpr (MODE == kByElement) {
#pragma unroll
      for (int i = 0; i < V; ++i) row[u * V + i] = (T)x.v[c][i];
    } else {
      Vec<T, V> y;
#pragma unroll
      for (int i = 0; i < V; ++i) y.e[i] = (T)x.v[c][i];
      *reinterpret_cast<Vec<T, V>*>(row + u * V) = y;
    }
  }
}

// The partners of a lane's channels, a byte each.
template <int C, int V>
struct Partners {
  uint32_t b[C * V / 4];
  template <int G>
  __device__ __forceinline__ void find(const uint8_t* partner, int j, int pieces) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < V; i += 4)
        b[(c * V + i) / 4] = *reinterpret_cast<const uint32_t*>(partner + min(j + c * G, pieces - 1) * V + i);
  }
};

// y sin, 0 where the sine is 0 whatever y holds: a channel that does not turn, or not yet, takes
// nothing of its partner, an infinity or a NaN least of all. (Comparing channels instead
// keeps a lane's results over the heads: 121 to 137 registers for 117, and the gradient of
// 18432 tokens takes up to 167 us for 138.)
__device__ __forceinline__ float of_partner(float y, float sine) {
  float z;
  asm("v_mul_legacy_f32 %0, %1, %2" : "=v"(z) : "v"(y), "v"(sine));
  return z;
}

// x[c] cos + x[partner] sin (with BACK - : turned back) for a head. In kApart and
// kByElement `room` is the head's own D floats of LDS; its lanes are in one wave, whose
// LDS operations are done in order.
template <int C, int V, int G, int MODE, bool BACK>
__device__ __forceinline__ void turn_head(const float2* cs, const Partners<C, V>& w, float* room,
                                          int j, int pieces, Vals<C, V>& x) {
  if constexpr (MODE != kAdjacent) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (j + c * G < pieces)
#pragma unroll
        for (int i = 0; i < V; ++i) room[(j + c * G) * V + i] = x.v[c][i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int at = min(j + c * G, pieces - 1) * V;
    float y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (MODE == kAdjacent)
        y[i] = x.v[c][i ^ 1];
      else
        y[i] = room[(w.b[(c * V + i) / 4] >> (8 * (i % 4))) & 255];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (MODE == kAdjacent) {
        const float2 t = cs[(at + i) / 2];
        const float z = of_partner(y[i], t.y);
        x.v[c][i] = __builtin_fmaf(x.v[c][i], t.x, (i % 2 == 0) != BACK ? -z : z);
      } else {
        const float2 t = cs[at + i];
        const float z = of_partner(y[i], t.y);
        x.v[c][i] = __builtin_fmaf(x.v[c][i], t.x, BACK ? -z : z);
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

// Cosines and sines of `n` tokens from `tok0` on into turn[token][pair], or signed into
// turn[token][channel].
template <int MODE>
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
    if constexpr (MODE == kAdjacent) {
      turn[i] = cs;
    } else {
      turn[t * a.D + c1] = make_float2(cs.x, -cs.y);
      turn[t * a.D + c2] = cs;
    }
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

// The gammas, and the partner of each channel.
__device__ __forceinline__ void fetch_tables(const HeadsArgs& a, float (*gamma)[kMaxDim],
                                             uint8_t* partner) {
  for (int i = threadIdx.x; i < 2 * a.D; i += kThreads) {
    const int part = i / a.D, c = i - part * a.D;
    gamma[part][c] = a.gamma[part] ? read_w(a.gamma[part], a.w_bf16, c) : 1.0f;
  }
  for (int p = threadIdx.x; p < a.D / 2; p += kThreads) {
    int c1, c2;
    pair_channels(a, p, c1, c2);
    partner[c1] = c2;
    partner[c2] = c1;
  }
}

// ----------------------------------------------------------------- forward ----

template <typename XT, typename YT, int G, int C, int MODE>
__global__ __launch_bounds__(kThreads) void k_heads(HeadsArgs a) {
  constexpr int V = kV<XT>, kGroups = kThreads / G;
  constexpr int kRoom = C * G * V + 1;  // an odd step from head to head: other banks
  __shared__ __attribute__((aligned(16))) float gamma[2][kMaxDim];
  __shared__ __attribute__((aligned(16))) float rooms[MODE == kAdjacent ? 4 : kGroups * kRoom];
  __shared__ __attribute__((aligned(4))) uint8_t partner[kMaxDim];
  __shared__ Starts starts[kMaxTokens];
  extern __shared__ __attribute__((aligned(16))) float2 turn[];  // [tokens][D]
  const int tid = threadIdx.x, group = tid / G, j = tid % G, pieces = a.D / V;
  const int turns = MODE == kAdjacent ? a.D / 2 : a.D;  // of a token
  float* const room = rooms + (MODE == kAdjacent ? 0 : group * kRoom);
  const int64_t all = (int64_t)a.B * a.L, tok0 = (int64_t)blockIdx.x * a.tokens;
  const int n = (int)(all - tok0 < a.tokens ? all - tok0 : a.tokens);
  const int heads = a.heads[0] + a.heads[1] + a.heads[2], rows = n * heads;
  find_starts(a, starts, tok0, n);
  __syncthreads();
  const auto row_in = [&](int r) {
    const int t = r / heads;
    return reinterpret_cast<const XT*>(a.x) + starts[t].x + (r - t * heads) * a.D;
  };
  Vals<C, V> v, next;
  load<XT, C, V, G, MODE>(row_in(min(group, rows - 1)), j, pieces, group < rows, next);
  fetch_tables(a, gamma, partner);
  form_turns<MODE>(a, turn, tok0, n);
  __syncthreads();
  Partners<C, V> with;
  with.template find<G>(partner, j, pieces);
  for (int r = group; r < rows; r += kGroups) {
    v = next;
    const int rn = r + kGroups;
    load<XT, C, V, G, MODE>(row_in(min(rn, rows - 1)), j, pieces, rn < rows, next);
    const int t = r / heads;
    int hd = r - t * heads;
    const int part = hd < a.heads[0] ? 0 : hd < a.heads[0] + a.heads[1] ? 1 : 2;
    if (part == 1) hd -= a.heads[0];
    if (part == 2) hd -= a.heads[0] + a.heads[1];
    if (part < 2) {
      if (a.rms) {
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < V; ++i) sum = __builtin_fmaf(v.v[c][i], v.v[c][i], sum);
        const float rstd = rsqrtf(head_sum<G>(sum) / (float)a.D + a.eps);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int at = min(j + c * G, pieces - 1) * V;
#pragma unroll
          for (int i = 0; i < V; ++i) v.v[c][i] *= rstd * gamma[part][at + i];
        }
      }
      if (a.n_axes) turn_head<C, V, G, MODE, false>(turn + t * turns, with, room, j, pieces, v);
    }
    store<YT, C, V, G, MODE>(reinterpret_cast<YT*>(a.y[part].p) + starts[t].y[part] +
                                 hd * a.y[part].head,
                             j, pieces, v);
  }
}

// ---------------------------------------------------------------- backward ----

// blockIdx.y says which part (q, k, v) a workgroup works for, so that a lane keeps
// one sum of dgamma; it walks over the tokens in steps of gridDim.x tiles.
template <typename XT, typename YT, int G, int C, int MODE>
__global__ __launch_bounds__(kThreads) void k_heads_grad(HeadsArgs a) {
  constexpr int V = kV<XT>, kGroups = kThreads / G;
  constexpr int kRoom = C * G * V + 1;  // an odd step from head to head: other banks
  __shared__ __attribute__((aligned(16))) float gamma[2][kMaxDim];
  __shared__ __attribute__((aligned(16))) float rooms[MODE == kAdjacent ? 4 : kGroups * kRoom];
  __shared__ __attribute__((aligned(4))) uint8_t partner[kMaxDim];
  __shared__ float sums[kThreads / 64][kMaxDim];
  __shared__ Starts starts[kMaxTokens];
  extern __shared__ __attribute__((aligned(16))) float2 turn[];
  const int tid = threadIdx.x, group = tid / G, j = tid % G, pieces = a.D / V;
  const int turns = MODE == kAdjacent ? a.D / 2 : a.D;  // of a token
  float* const room = rooms + (MODE == kAdjacent ? 0 : group * kRoom);
  const int part = blockIdx.y, heads = a.heads[part];
  const int64_t all = (int64_t)a.B * a.L;
  const int head0 = part == 0 ? 0 : part == 1 ? a.heads[0] : a.heads[0] + a.heads[1];
  fetch_tables(a, gamma, partner);
  __syncthreads();
  Partners<C, V> with;
  with.template find<G>(partner, j, pieces);
  Vals<C, V> dg;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < V; ++i) dg.v[c][i] = 0.0f;
  const ql_heads_view& y = a.y[part];
  const int64_t step = (int64_t)gridDim.x * a.tokens;
  for (int64_t tok0 = (int64_t)blockIdx.x * a.tokens; tok0 < all && heads > 0; tok0 += step) {
    const int n = (int)(all - tok0 < a.tokens ? all - tok0 : a.tokens), rows = n * heads;
    __syncthreads();  // the turns before have been read
    find_starts(a, starts, tok0, n);
    if (part < 2) form_turns<MODE>(a, turn, tok0, n);
    __syncthreads();
    for (int r = group; r < rows; r += kGroups) {
      const int t = r / heads, hd = r - t * heads;
      Vals<C, V> x, d;
      load<YT, C, V, G, MODE>(reinterpret_cast<const YT*>(y.p) + starts[t].y[part] + hd * y.head, j,
                              pieces, true, d);
      if (part < 2) {
        if (a.rms)
          load<XT, C, V, G, MODE>(reinterpret_cast<const XT*>(a.x) + starts[t].x +
                                      (head0 + hd) * a.D, j, pieces, true, x);
        if (a.n_axes) turn_head<C, V, G, MODE, true>(turn + t * turns, with, room, j, pieces, d);
        if (a.rms) {
          float s2 = 0.0f, st = 0.0f;
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const int at = min(j + c * G, pieces - 1) * V;
#pragma unroll
            for (int i = 0; i < V; ++i) {
              s2 = __builtin_fmaf(x.v[c][i], x.v[c][i], s2);
              st = __builtin_fmaf(d.v[c][i] * gamma[part][at + i], x.v[c][i], st);
            }
          }
          s2 = head_sum<G>(s2);
          st = head_sum<G>(st);
          const float rstd = rsqrtf(s2 / (float)a.D + a.eps);
          const float f = rstd * rstd * (st / (float)a.D);
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const int at = min(j + c * G, pieces - 1) * V;
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float dn = d.v[c][i], xv = x.v[c][i];
              dg.v[c][i] = __builtin_fmaf(dn, xv * rstd, dg.v[c][i]);
              d.v[c][i] = rstd * __builtin_fmaf(dn, gamma[part][at + i], -(xv * f));
            }
          }
        }
      }
      store<XT, C, V, G, MODE>(reinterpret_cast<XT*>(a.dx) + starts[t].dx + (head0 + hd) * a.D, j,
                               pieces, d);
    }
  }
  if (!a.part || part == 2) return;
  // lanes of the same pieces, then waves
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float v = dg.v[c][i];
      if constexpr (G <= 4) v += __shfl_xor(v, 4);
      if constexpr (G <= 8) v += __shfl_xor(v, 8);
      v += __shfl_xor(v, 16);
      v += __shfl_xor(v, 32);
      if ((tid & 63) < G && j + c * G < pieces) sums[tid >> 6][(j + c * G) * V + i] = v;
    }
  __syncthreads();
  for (int i = tid; i < a.D; i += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) v += sums[w][i];
    a.part[((int64_t)part * gridDim.x + blockIdx.x) * a.D + i] = v;
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
  if (a.w_bf16)
    reinterpret_cast<bf16*>(a.dgamma[part])[i] = (bf16)(float)sum;
  else
    reinterpret_cast<float*>(a.dgamma[part])[i] = (float)sum;
}

// ------------------------------------------------------------------ launch ----

// How a call's rows are read.
int mode_of(const HeadsArgs& a) { return !a.vec ? kByElement : a.halves && a.n_axes ? kApart : kAdjacent; }

template <typename XT, typename YT, int G, int C>
hipError_t run(const HeadsArgs& a, bool grad, dim3 grid, hipStream_t s) {
  const int mode = mode_of(a);
  const size_t lds = (size_t)a.tokens * (mode == kAdjacent ? a.D / 2 : a.D) * sizeof(float2);
  // the kernels' own LDS and the turns of kMaxTokens tokens pass 64 KB at long heads of few
  constexpr int most = kMaxTokens * kMaxDim * (int)sizeof(float2);
  hipError_t e = hipSuccess;
#define QL_HEADS_MODE(M)                                                              \
  if (mode == M) {                                                                    \
    if (grad) {                                                                       \
      if (M != kAdjacent) e = allow_lds<&k_heads_grad<XT, YT, G, C, M>, most>();      \
      if (e == hipSuccess) k_heads_grad<XT, YT, G, C, M><<<grid, kThreads, lds, s>>>(a); \
    } else {                                                                          \
      if (M != kAdjacent) e = allow_lds<&k_heads<XT, YT, G, C, M>, most>();           \
      if (e == hipSuccess) k_heads<XT, YT, G, C, M><<<grid, kThreads, lds, s>>>(a);   \
    }                                                                                 \
  }
  QL_HEADS_MODE(kAdjacent)
  QL_HEADS_MODE(kApart)
  QL_HEADS_MODE(kByElement)
#undef QL_HEADS_MODE
  return e == hipSuccess ? hipGetLastError() : e;
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

// LDS of k_heads but for the turns: the gammas, the partners, the tokens' starts, and a room for
// each head where partners trade places.
int fixed_lds(const HeadsArgs& a, int lanes) {
  const int padded = a.D == 64 || a.D == 128 ? a.D : (a.D + 31) / 32 * 32;
  const int rooms = mode_of(a) == kAdjacent ? 16 : kThreads / lanes * (padded + 1) * 4;
  return 2 * kMaxDim * 4 + kMaxDim + kMaxTokens * (int)sizeof(Starts) + 64 + rooms;
}

// Tokens of a workgroup: enough rows for four passes of its lanes, unless that leaves fewer
// workgroups than fill the chip; forward no more than leave LDS for two workgroups on a compute
// unit (three heads of 160 a token, pairs in halves, bf16, 120000 tokens: 251 us with the 32 tokens
// that take 87 KB, 164 with the 27 that take 80, 182 with 14 and 64). The gradient, whose workgroups
// take one part's heads each and walk over many tokens, keeps them (502, 564, 828).
int tokens_of(const HeadsArgs& a, int64_t all, int heads, bool grad) {
  const int lanes = a.x_bf16 ? lanes_of<bf16>(a.D) : lanes_of<float>(a.D), groups = kThreads / lanes;
  int t = 1;
  while (t < kMaxTokens && t * heads < 4 * groups &&
         (t * heads < groups || all / (2 * t) >= 1024))
    t *= 2;
  const int each = (mode_of(a) == kAdjacent ? a.D / 2 : a.D) * (int)sizeof(float2);
  const int most = (80 * 1024 - fixed_lds(a, lanes)) / each;
  return grad || t < most ? t : most;
}

}  // namespace

int heads_grad_groups(int64_t tokens) {
  return (int)(tokens < 512 ? (tokens < 1 ? 1 : tokens) : 512);
}

hipError_t launch_heads(const HeadsArgs& args, hipStream_t s) {
  HeadsArgs a = args;
  const int64_t all = (int64_t)a.B * a.L;
  a.tokens = tokens_of(a, all, a.heads[0] + a.heads[1] + a.heads[2], false);
  return go(a, false, dim3((unsigned)((all + a.tokens - 1) / a.tokens)), s);
}

hipError_t launch_heads_grad(const HeadsArgs& args, hipStream_t s) {
  HeadsArgs a = args;
  const int64_t all = (int64_t)a.B * a.L;
  if (all > 0) {
    const int most = a.heads[0] > a.heads[1] ? a.heads[0] : a.heads[1];
    a.tokens = tokens_of(a, all, most > a.heads[2] ? most : a.heads[2], true);
    const hipError_t e = go(a, true, dim3((unsigned)a.groups, 3), s);
    if (e != hipSuccess) return e;
  }
  if (!a.dgamma[0] && !a.dgamma[1]) return hipSuccess;
  if (all == 0) a.groups = 0;
  k_heads_gamma<<<dim3((a.D + 31) / 32, 2), 1024, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ql
