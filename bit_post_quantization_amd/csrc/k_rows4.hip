// Few rows against 4-bit weights with a scale for each group of input channels.
//
//   Y[m,n] = bias[n] + sum_g scale[n,g] sum_{k in g} code[n,k] act(X[m,k])
//
// A modulation linear reads a conditioning vector an image: the weights are most of what
// moves (N K / 2 bytes), so the kernel is built to read them once, in order, with many
// loads in flight. The matrix cores take 16 output channels by 32 inputs of codes as
// rows and 16 rows of X as columns (v_mfma_f32_16x16x32_bf16); with 16 columns or
// fewer the unpacking of a code (about two operations) is what they wait for, and it is
// done once for all rows. A 4-bit integer is exact in bf16, and act(X) is split
// into three bf16 terms that hold its 24 bits (one for bf16 X as it is), so products are
// exact and sums fp32; a step's sum is multiplied by its group's scale in fp32.
//
// A workgroup of eight waves has NT tiles of 16 channels and all rows; its waves share
// out the steps of 32 inputs, and join their sums in LDS at the end.
#include "ql_block.h"
#include "ql_device.h"

namespace ql {

namespace {

typedef __bf16 bf16;
typedef float v4f __attribute__((ext_vector_type(4)));
typedef bf16 v8h __attribute__((ext_vector_type(8)));
typedef bf16 v4h __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kMaxBlocks = 3;       // 16-row blocks of a workgroup
constexpr int kXBytes = 64 * 1024;  // of LDS for act(X): two workgroups a compute unit

// Eight codes of a word (nibble j: input j), as bf16.
__device__ __forceinline__ v8h unpack(uint32_t w) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = (float)((int)(w << (28 - 4 * j)) >> 28);
  uint32_t p[4];  // small integers: the upper halves are the values
#pragma unroll
  for (int j = 0; j < 4; ++j)
    p[j] = __builtin_amdgcn_perm(__float_as_uint(f[2 * j + 1]), __float_as_uint(f[2 * j]),
                                 0x07060302u);
  return __builtin_bit_cast(v8h, v4u{p[0], p[1], p[2], p[3]});
}

// x / (1 + exp(-x)) to about two units in the last place: the exponent's rounding is put
// back (-x log2 e in two parts), v_exp_f32 and v_rcp_f32 are good to one.
__device__ __forceinline__ float silu(float x) {
  constexpr float kHi = 1.44269502162933350f, kLo = 1.92596299112661746e-8f;
  const float t = -x * kHi;
  const float lo = __builtin_fmaf(-x, kHi, -t) - x * kLo;
  const float e = __builtin_amdgcn_exp2f(t);
  const float y = x * __builtin_amdgcn_rcpf(1.0f + __builtin_fmaf(e * 0.6931472f, lo, e));
  // exp overflows, or lo is not a number: the limits
  return t >= 128.0f ? (x == -INFINITY ? NAN : -0.0f) : t <= -128.0f ? x : y;
}


template <int NT, int MB, int TERMS>
__global__ __launch_bounds__(kThreads) void k_rows4(Rows4Args a, int fill) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  bf16* const xs = reinterpret_cast<bf16*>(smem);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), r16 = lane & 15, quad = lane >> 4;
  const int tile0 = blockIdx.x * NT, m0 = blockIdx.y * 16 * MB, sp = blockIdx.z;
  const int rows = min(a.M - m0, 16 * MB);
  const int per = (a.steps + a.splits - 1) / a.splits;
  const int s0 = min(sp * per, a.steps), s1 = min(s0 + per, a.steps);
  const int ld = fill * 32 + 8, plane = rows * ld;  // an odd number of 16-byte pieces
  const int share = (fill + kWaves - 1) / kWaves;   // steps of a wave in a filling
  v4f acc[NT][MB];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[t][b] = v4f{0, 0, 0, 0};

  constexpr int U = 4;  // steps whose loads are in flight
  uint32_t code[NT][U];
  v4f scale[NT][U];
  const auto fetch = [&](int first, int end) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = min(first + u, max(end - 1, 0));
      const int g = s / a.group_steps;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int tile = min(tile0 + t, a.tiles - 1);
        code[t][u] = a.codes[((int64_t)tile * a.steps + s) * 64 + lane];
        const int64_t at = ((int64_t)tile * a.groups + g) * 16 + 4 * quad;
        if (a.s_bf16) {
          const v4h v = *reinterpret_cast<const v4h*>(reinterpret_cast<const bf16*>(a.scales) + at);
#pragma unroll
          for (int e = 0; e < 4; ++e) scale[t][u][e] = (float)v[e];
        } else {
          scale[t][u] = *reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(a.scales) + at);
        }
      }
    }
  };

  for (int c0 = s0; c0 < s1; c0 += fill) {
    const int c1 = min(c0 + fill, s1);
    const int b = min(c0 + wave * share, c1), e = min(b + share, c1);
    fetch(b, e);
    if (c0 > s0) __syncthreads();  // the filling before has been read
    // act(X) of the filling, four inputs a thread at a time
    const int quads = (c1 - c0) * 8;
    for (int i = tid; i < rows * quads; i += kThreads) {
      const int r = i / quads, k4 = i - r * quads, k = c0 * 32 + 4 * k4;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (k < a.K) {  // K is a multiple of 16
        const int64_t at = (int64_t)(m0 + r) * a.ldx + k;
        if (a.x_bf16) {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = (float)reinterpret_cast<const bf16*>(a.X)[at + j];
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = reinterpret_cast<const float*>(a.X)[at + j];
        }
      }
      if (a.silu) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = silu(v[j]);
      }
#pragma unroll
      for (int t = 0; t < TERMS; ++t) {
        v4h h;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[j] = (bf16)v[j];
          v[j] -= (float)h[j];
        }
        *reinterpret_cast<v4h*>(xs + t * plane + r * ld + 4 * k4) = h;
      }
    }
    __syncthreads();
    for (int s = b; s < e; s += U) {
      uint32_t w[NT][U];
      v4f sc[NT][U];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          w[t][u] = code[t][u];
          sc[t][u] = scale[t][u];
        }
      if (s + U < e) fetch(s + U, e);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (s + u >= e) break;
        v8h x[MB][TERMS];
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
          for (int t = 0; t < TERMS; ++t)
            x[m][t] = *reinterpret_cast<const v8h*>(
                xs + t * plane + min(16 * m + r16, rows - 1) * ld + (s + u - c0) * 32 + 8 * quad);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const v8h c = unpack(w[t][u]);
#pragma unroll
          for (int m = 0; m < MB; ++m) {
            v4f sum = {0, 0, 0, 0};
#pragma unroll
            for (int p = TERMS - 1; p >= 0; --p)  // the small terms first
              sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(c, x[m][p], sum, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[t][m][i] = __builtin_fmaf(sum[i], sc[t][u][i], acc[t][m][i]);
          }
        }
      }
    }
  }
  // the waves' sums: box[wave][block][row][channel of the workgroup's]
  __syncthreads();
  float* const box = reinterpret_cast<float*>(smem);
  constexpr int kCh = NT * 16, kOne = MB * 16 * kCh;
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
      *reinterpret_cast<v4f*>(box + wave * kOne + (16 * m + r16) * kCh + 16 * t + 4 * quad) =
          acc[t][m];
  __syncthreads();
  for (int i = tid; i < rows * kCh; i += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += box[w * kOne + i];
    const int r = i / kCh, n = tile0 * 16 + i % kCh;
    if (n >= a.N) continue;
    if (a.splits > 1)
      a.part[((int64_t)sp * a.M + m0 + r) * a.N + n] = v;
    else
      a.Y[(int64_t)(m0 + r) * a.ldy + n] = a.bias ? v + a.bias[n] : v;
  }
}

__global__ __launch_bounds__(256) void k_rows4_join(Rows4Args a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)a.M * a.N;
  if (i >= all) return;
  float v = 0.0f;
  for (int s = 0; s < a.splits; ++s) v += a.part[s * all + i];
  const int m = (int)(i / a.N), n = (int)(i - (int64_t)m * a.N);
  a.Y[m * a.ldy + n] = a.bias ? v + a.bias[n] : v;
}

// Rows and channels of a workgroup: as many tiles as leave one workgroup a compute unit
// (act(X) is formed again by each), 48 rows where there are more than 16.
int blocks_of(int M) { return M <= 16 ? 1 : M <= 32 ? 2 : kMaxBlocks; }
int tiles_of(int M, int tiles) {
  const int groups = (M + 16 * blocks_of(M) - 1) / (16 * blocks_of(M));
  return M > 16 || (int64_t)tiles * groups < 512 ? (M > 16 ? 2 : 1) : tiles < 1024 ? 2 : 4;
}

template <int NT, int MB, int TERMS>
hipError_t run(const Rows4Args& a, hipStream_t s) {
  const int rows = a.M < 16 * MB ? a.M : 16 * MB;
  const int per = (a.steps + a.splits - 1) / a.splits;
  int most = (kXBytes / (rows * TERMS * 2) - 8) / 32 / kWaves * kWaves;
  if (most < kWaves) most = kWaves;
  const int fills = (per + most - 1) / most;
  int fill = (per + fills - 1) / fills;
  fill = (fill + kWaves - 1) / kWaves * kWaves;
  const int x = rows * TERMS * 2 * (fill * 32 + 8), box = kWaves * NT * MB * 1024;
  const int groups = (a.M + 16 * MB - 1) / (16 * MB);
  const dim3 grid((a.tiles + NT - 1) / NT, groups, a.splits);
  const int lds = x > box ? x : box;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_rows4<NT, MB, TERMS>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  k_rows4<NT, MB, TERMS><<<grid, kThreads, lds, s>>>(a, fill);
  return hipGetLastError();
}

// ------------------------------------------------------------------ layout ----

struct PackArgs {
  const int8_t* codes;    // [N, K]
  const void* scales;     // [N, groups]
  const void* W;          // quantize: [N, K]
  uint32_t* packed;
  void* packed_scales;
  int N, K, steps, tiles, groups, group;
  bool s_bf16, w_bf16;
};

__device__ __forceinline__ float w_at(const PackArgs& a, int64_t i) {
  return a.w_bf16 ? (float)reinterpret_cast<const bf16*>(a.W)[i]
                  : reinterpret_cast<const float*>(a.W)[i];
}

// One word a thread.
__global__ __launch_bounds__(256) void k_rows4_pack(PackArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.tiles * a.steps * 64) return;
  const int lane = (int)(i % 64), step = (int)(i / 64 % a.steps), tile = (int)(i / 64 / a.steps);
  const int n = tile * 16 + lane % 16, k = step * 32 + 8 * (lane / 16);
  uint32_t w = 0;
  if (n < a.N && k < a.K)  // K is a multiple of 16
    for (int j = 0; j < 8; ++j)
      w |= ((uint32_t)a.codes[(int64_t)n * a.K + k + j] & 15u) << (4 * j);
  a.packed[i] = w;
}

// One scale a thread; in packed order.
__global__ __launch_bounds__(256) void k_rows4_pack_scales(PackArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.tiles * a.groups * 16) return;
  const int r = (int)(i % 16), g = (int)(i / 16 % a.groups), tile = (int)(i / 16 / a.groups);
  const int n = tile * 16 + r;
  const int64_t at = (int64_t)n * a.groups + g;
  if (a.s_bf16)
    reinterpret_cast<bf16*>(a.packed_scales)[i] =
        n < a.N ? reinterpret_cast<const bf16*>(a.scales)[at] : (bf16)0.0f;
  else
    reinterpret_cast<float*>(a.packed_scales)[i] =
        n < a.N ? reinterpret_cast<const float*>(a.scales)[at] : 0.0f;
}

// One group of one channel a thread: its scale, then its codes by that scale.
__global__ __launch_bounds__(256) void k_rows4_quantize(PackArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.tiles * a.groups * 16) return;
  const int r = (int)(i % 16), g = (int)(i / 16 % a.groups), tile = (int)(i / 16 / a.groups);
  const int n = tile * 16 + r, k0 = g * a.group, k1 = min(k0 + a.group, a.K);
  float top = 0.0f;
  if (n < a.N)
    for (int k = k0; k < k1; ++k) top = fmaxf(top, fabsf(w_at(a, (int64_t)n * a.K + k)));
  float s = top / 7.0f;
  if (a.s_bf16) {
    const bf16 b = (bf16)s;
    reinterpret_cast<bf16*>(a.packed_scales)[i] = b;
    s = (float)b;
  } else {
    reinterpret_cast<float*>(a.packed_scales)[i] = s;
  }
  for (int k = k0; k < k0 + a.group && k < a.steps * 32; k += 8) {
    uint32_t w = 0;
    for (int j = 0; j < 8; ++j) {
      int c = 0;
      if (n < a.N && k + j < a.K && s > 0.0f)
        c = (int)fminf(fmaxf(rintf(w_at(a, (int64_t)n * a.K + k + j) / s), -7.0f), 7.0f);
      w |= ((uint32_t)c & 15u) << (4 * j);
    }
    a.packed[((int64_t)tile * a.steps + k / 32) * 64 + 16 * (k % 32 / 8) + r] = w;
  }
}

// Four codes or one scale a thread.
__global__ __launch_bounds__(256) void k_rows4_unpack(PackArgs a, int8_t* codes, void* scales) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (codes && i < (int64_t)a.N * (a.K / 4)) {
    const int n = (int)(i / (a.K / 4)), k = (int)(i % (a.K / 4)) * 4;
    const uint32_t w = a.packed[((int64_t)(n / 16) * a.steps + k / 32) * 64 + 16 * (k % 32 / 8) + n % 16] >>
                       (4 * (k % 8));
    for (int j = 0; j < 4; ++j)
      codes[(int64_t)n * a.K + k + j] = (int8_t)((int)(w << (28 - 4 * j)) >> 28);
  }
  if (scales && i < (int64_t)a.N * a.groups) {
    const int n = (int)(i / a.groups), g = (int)(i % a.groups);
    const int64_t at = ((int64_t)(n / 16) * a.groups + g) * 16 + n % 16;
    if (a.s_bf16)
      reinterpret_cast<bf16*>(scales)[i] = reinterpret_cast<const bf16*>(a.packed_scales)[at];
    else
      reinterpret_cast<float*>(scales)[i] = reinterpret_cast<const float*>(a.packed_scales)[at];
  }
}

PackArgs pack_args(const ql_rows4& d, const void* packed) {
  const Rows4Layout l = rows4_layout(d);
  PackArgs a{};
  char* p = reinterpret_cast<char*>(const_cast<void*>(packed));
  a.packed = reinterpret_cast<uint32_t*>(p);
  a.packed_scales = p + l.scales;
  a.N = d.N;
  a.K = d.K;
  a.steps = l.steps;
  a.tiles = l.tiles;
  a.groups = l.groups;
  a.group = d.group;
  a.s_bf16 = d.s_dtype == QL_BF16;
  return a;
}

unsigned blocks(int64_t n) { return (unsigned)((n + 255) / 256); }

}  // namespace

Rows4Layout rows4_layout(const ql_rows4& d) {
  Rows4Layout l;
  l.tiles = (d.N + 15) / 16;
  l.steps = (d.K + 31) / 32;
  l.groups = (d.K + d.group - 1) / d.group;
  l.scales = (int64_t)l.tiles * l.steps * 256;
  l.bytes = l.scales + (int64_t)l.tiles * l.groups * 16 * (d.s_dtype == QL_BF16 ? 2 : 4);
  return l;
}

int rows4_splits(int M, int N, int K) {
  const int tiles = (N + 15) / 16, steps = (K + 31) / 32, NT = tiles_of(M, tiles);
  const int64_t groups = (M + 16 * blocks_of(M) - 1) / (16 * blocks_of(M));
  const int64_t base = (tiles + NT - 1) / NT * groups;
  if (base > 96 || steps < 64) return 1;
  int64_t n = 256 / base;
  if (n > steps / 32) n = steps / 32;
  return (int)(n < 1 ? 1 : n > 16 ? 16 : n);
}

hipError_t launch_rows4(const Rows4Args& a, hipStream_t s) {
  const bool one = a.x_bf16 && !a.silu;
  const int NT = tiles_of(a.M, a.tiles), MB = blocks_of(a.M);
  hipError_t e = hipErrorInvalidValue;
#define QL_ROWS4(T, B) \
  if (NT == T && MB == B) e = one ? run<T, B, 1>(a, s) : run<T, B, 3>(a, s);
  QL_ROWS4(1, 1)
  QL_ROWS4(2, 1)
  QL_ROWS4(4, 1)
  QL_ROWS4(2, 2)
  QL_ROWS4(2, 3)
#undef QL_ROWS4
  if (e != hipSuccess || a.splits == 1) return e;
  k_rows4_join<<<blocks((int64_t)a.M * a.N), 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_rows4_pack(const ql_rows4& d, const int8_t* codes, const void* scales,
                             void* packed, hipStream_t s) {
  PackArgs a = pack_args(d, packed);
  a.codes = codes;
  a.scales = scales;
  k_rows4_pack<<<blocks((int64_t)a.tiles * a.steps * 64), 256, 0, s>>>(a);
  k_rows4_pack_scales<<<blocks((int64_t)a.tiles * a.groups * 16), 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_rows4_quantize(const ql_rows4& d, const void* W, bool w_bf16, void* packed,
                                 hipStream_t s) {
  PackArgs a = pack_args(d, packed);
  a.W = W;
  a.w_bf16 = w_bf16;
  k_rows4_quantize<<<blocks((int64_t)a.tiles * a.groups * 16), 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_rows4_unpack(const ql_rows4& d, int8_t* codes, void* scales, hipStream_t s) {
  const PackArgs a = pack_args(d, d.packed);
  const int64_t n = (int64_t)a.N * (a.K / 4), m = (int64_t)a.N * a.groups;
  k_rows4_unpack<<<blocks(n > m ? n : m), 256, 0, s>>>(a, codes, scales);
  return hipGetLastError();
}

}  // namespace ql
