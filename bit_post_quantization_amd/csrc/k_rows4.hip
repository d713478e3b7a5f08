// Few rows against 4-bit weights with a scale for each group of input channels.
//
//   Y[m,n] = bias[n] + sum_g scale[n,g] sum_{k in g} code[n,k] act(X[m,k])
//
// A modulation linear reads a conditioning vector an image: the weights are most of what
// moves (N K / 2 bytes), so the kernel is built to read them once, in order, with many
// loads in flight, and to do little for each code. The product is one of integers:
// act(X) is written in fixed point, for each row and unit of 128 inputs 31 bits below
// the power of two above the largest value, as four signed 8-bit digits (t = x + 0x00808080, the
// bytes of t ^ 0x00808080; they hold up to 0x7f7f7f7f, so 30 bits where the value is within
// 0.4 % of that power). What that drops is at most 1.004 * 2^-31 of the unit's largest value,
// and nothing of values within 2^-6 of it. v_mfma_i32_16x16x64_i8 (x32 for groups of 32)
// multiplies 16 output channels' codes by 16 rows' digits exactly; codes go in as
// 16 times their value, so that eight of them take three operations (in bf16, with X in
// three terms, it was 28, and the rows' terms 6 bytes instead of 4). A group's four sums
// are joined in fp32 and scaled: 28 operations for 16 by 16 outputs.
//
// Measured: 2 rows, K 1152, N 6912: 5.6 us of kernel (latency); 8 rows, K 4096, N 24576: 21.4 us a
// call, of kernels 3-4 for the digits and 18-20 for the products, 2.5 TB/s in all: a wave asks for two
// of its four units' codes, and for the others only once the workgroup, the only one on its
// compute unit, has all rows' digits; 77 rows, K 4608, N 1151, groups of 32: 4 and 14 us, bound by
// the joining of its sums and latency. Beside one large input the digits of the others are coarser:
// against 64 bits, 8 rows, K 1152, N 4096, one input R times the rest whose codes are 0, outputs are off
// by 7e-8 of their size up to R = 100, 8e-8 at 1e3, 2e-7 at 4e3, 1.5e-6 at 3e4, 5e-5 at 1e6 (products
// in fp32: 3e-7).
//
// The waves of a workgroup share out the units of its NT tiles of 16 channels and join
// in LDS. The digits come from LDS where the rows fit: formed there by the workgroup, if
// they are few, else copied from what k_rows4_digits formed once; or else, and for
// more than 16 rows, from memory.
#include "ql_block.h"
#include "ql_device.h"

namespace ql {

namespace {

typedef __bf16 bf16;
typedef float v4f __attribute__((ext_vector_type(4)));
typedef bf16 v8h __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

constexpr int kWaves = 8, kThreads = 64 * kWaves;  // that share a tile's inputs
constexpr int kUnit = 128;
constexpr int kUnitBytes = 4 * kUnit;    // of a row's digits
constexpr int kXBytes = 144 * 1024;      // of LDS at most for digits

// Eight codes of a word (nibble j: input j) times 16: inputs 0 2 4 6, and 1 3 5 7.
__device__ __forceinline__ uint32_t even(uint32_t w) { return (w << 4) & 0xf0f0f0f0u; }
__device__ __forceinline__ uint32_t odd(uint32_t w) { return w & 0xf0f0f0f0u; }

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

// Eight inputs of a row, k a multiple of 8.
__device__ __forceinline__ void load_x(const Rows4Args& a, int m, int k, float (&v)[8]) {
  const int64_t at = m * a.ldx + k;
  if (a.x_bf16) {
    const bf16* p = reinterpret_cast<const bf16*>(a.X) + at;
    if (a.x_vec) {
      const v8h x = *reinterpret_cast<const v8h*>(p);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (float)x[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (float)p[j];
    }
  } else {
    const float* p = reinterpret_cast<const float*>(a.X) + at;
    if (a.x_vec) {
      const v4f x = *reinterpret_cast<const v4f*>(p), y = *reinterpret_cast<const v4f*>(p + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = x[j];
        v[4 + j] = y[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = p[j];
    }
  }
}

// Digits of eight inputs of one row by a group of 16 lanes that hold a unit of it: digit
// d of the inputs in the order of even() and odd() in out[d]. Returns what one unit of the fixed
// point, for the codes' 16 times their value, is worth (NaN where an input is not finite).
__device__ __forceinline__ float digits(const Rows4Args& a, int m, int k, uint2 (&out)[4]) {
  float v[8], top = 0.0f;
  bool finite = true;
  load_x(a, m, min(k, a.K - 8), v);  // K is a multiple of 16
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = k >= a.K ? 0.0f : a.silu ? silu(v[j]) : v[j];
    finite = finite && fabsf(v[j]) < INFINITY;
    top = fmaxf(top, fabsf(v[j]));
  }
  // largest value's exponent, one more where its mantissa, as 31 bits, is past 0x7f7f7f7f
  int t = finite ? (int)((__float_as_uint(top) + 0x010101u) >> 23) : 256;
  t = max(t, (int)xor_lane_u<1>(t));
  t = max(t, (int)xor_lane_u<2>(t));
  t = max(t, (int)xor_lane_u<4>(t));
  t = max(t, (int)xor_lane_u<8>(t));
  // largest value <= 0x7f7f7f7f 2^(e - 31), t = 256: not finite; worths are powers of two that
  // fp32 has, down to its smallest
  const int e = max(t, 12) - 126;
  uint32_t x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = (int)rintf(ldexpf(v[j], 31 - e));
    x[j] = ((uint32_t)i + 0x00808080u) ^ 0x00808080u;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // inputs 0 2 4 6, then 1 3 5 7: four words' bytes turned
    const uint32_t p = __builtin_amdgcn_perm(x[2 + h], x[h], 0x05010400u);      // a0 c0 a1 c1
    const uint32_t q = __builtin_amdgcn_perm(x[2 + h], x[h], 0x07030602u);      // a2 c2 a3 c3
    const uint32_t r = __builtin_amdgcn_perm(x[6 + h], x[4 + h], 0x05010400u);
    const uint32_t s = __builtin_amdgcn_perm(x[6 + h], x[4 + h], 0x07030602u);
    const uint32_t w[4] = {__builtin_amdgcn_perm(r, p, 0x05040100u), __builtin_amdgcn_perm(r, p, 0x07060302u),
                           __builtin_amdgcn_perm(s, q, 0x05040100u), __builtin_amdgcn_perm(s, q, 0x07060302u)};
#pragma unroll
    for (int d = 0; d < 4; ++d) (h ? out[d].y : out[d].x) = w[d];
  }
  return t == 256 ? NAN : ldexpf(1.0f, e - 35);
}

// LDS for rows' digits: whole kilobytes, as they are copied.
__host__ __device__ constexpr int digit_bytes(int rows, int units) {
  return (rows * units * kUnitBytes + 1023) / 1024 * 1024;
}

// Place of the digits of inputs 8 q + 32 (2 pair + half) .. + 7 of a unit: 16-byte pieces
// [unit][pair][digit][row][q], each the two halves' eight.
__device__ __forceinline__ int digit_at(int unit, int pair, int d, int row, int q, int rows) {
  return (((unit * 2 + pair) * 4 + d) * rows + row) * 4 + q;
}

// Digits and worths of all rows, in blocks of 16 (the last one may be short), each as
// digit_at lays it out; worths [row][unit]. 16 lanes a row's unit.
__global__ __launch_bounds__(256) void k_rows4_digits(Rows4Args a) {
  // a row a blockIdx.y, unit by unit: neighbouring inputs
  const int m = blockIdx.y + 32768 * blockIdx.z, unit = blockIdx.x * 16 + (threadIdx.x >> 4), l = threadIdx.x & 15;
  if (unit >= a.units || m >= a.M) return;
  uint2 d[4];
  const float f = digits(a, m, unit * kUnit + 8 * l, d);
  const int block = m / 16, rows = min(16, a.M - block * 16);
  char* base = a.digits + (int64_t)block * 16 * a.units * kUnitBytes;
  const int step = l / 4;
#pragma unroll
  for (int n = 0; n < 4; ++n)
    *reinterpret_cast<uint2*>(base + digit_at(unit, step / 2, n, m % 16, l % 4, rows) * 16 + 8 * (step % 2)) = d[n];
  if (l == 0) a.worths[(int64_t)m * a.units + unit] = f;
}

enum { kForm = 0, kCopy = 1, kRead = 2 };  // where a workgroup's digits come from

// Codes and scales of one unit of NT tiles: GS steps of 32 inputs to a group.
template <int NT, int GS, typename S>
struct Unit {
  typedef S v4s __attribute__((ext_vector_type(4)));
  v4u code[NT];
  v4s scale[NT][4 / GS];
  __device__ __forceinline__ void fetch(const Rows4Args& a, int tile0, int unit, int lane) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t at = (int64_t)min(tile0 + t, a.tiles - 1) * a.units + unit;
      code[t] = a.codes[at * 64 + lane];
#pragma unroll
      for (int g = 0; g < 4 / GS; ++g) {
        const int64_t sc = (at * (4 / GS) + g) * 16 + 4 * (lane >> 4);
        scale[t][g] = *reinterpret_cast<const v4s*>(reinterpret_cast<const S*>(a.scales) + sc);
      }
    }
  }
};

template <int NT, int MB, int GS, int SRC, typename S>
__global__ __launch_bounds__(kThreads) void k_rows4(Rows4Args a) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), r16 = lane & 15, quad = lane >> 4;
  const int tile0 = blockIdx.x * NT, block0 = blockIdx.y * MB;
  const int rows = min(a.M - block0 * 16, 16 * MB);
  // units, dealt in turn to the waves and to the workgroups that share the tiles
  const int step = kWaves * a.splits, first = blockIdx.z * kWaves + wave;
  Unit<NT, GS, S> x, y;
  if (first < a.units) x.fetch(a, tile0, first, lane);
  if (first + step < a.units) y.fetch(a, tile0, first + step, lane);

  float* const worths = reinterpret_cast<float*>(smem + (SRC == kRead ? 0 : digit_bytes(rows, a.units)));
  if constexpr (SRC == kForm) {
    for (int job = tid >> 4; job < rows * a.units; job += kThreads / 16) {
      const int m = job / a.units, unit = job - m * a.units, l = tid & 15;
      uint2 d[4];
      const float f = digits(a, m, unit * kUnit + 8 * l, d);
#pragma unroll
      for (int n = 0; n < 4; ++n)
        *reinterpret_cast<uint2*>(smem + digit_at(unit, l / 8, n, m, l % 4, rows) * 16 + 8 * (l / 4 % 2)) = d[n];
      if (l == 0) worths[job] = f;
    }
  } else if constexpr (SRC == kCopy) {
    // straight into LDS, a kilobyte a wave at a time; past the end come zeros
    const __amdgpu_buffer_rsrc_t from =
        __builtin_amdgcn_make_buffer_rsrc(a.digits, 0, rows * a.units * kUnitBytes, 0x00020000);
    for (int i = wave * 1024; i < rows * a.units * kUnitBytes; i += kThreads * 16)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void*)(smem + i), 16, i + lane * 16, 0, 0, 0);
    for (int i = tid; i < rows * a.units; i += kThreads) worths[i] = a.worths[i];
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
  if constexpr (SRC != kRead) __syncthreads();

  v4f acc[NT][MB];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int m = 0; m < MB; ++m) acc[t][m] = v4f{0, 0, 0, 0};
  // Digits of block m for a unit. From memory they come one block ahead of their use.
  const auto get = [&](int unit, int m, v4u (&d)[2][4]) {
    const v4u* from = reinterpret_cast<const v4u*>(smem);
    int row = min(16 * m + r16, rows - 1), in_block = rows;
    if constexpr (SRC == kRead) {
      const int block = min(block0 + m, (a.M - 1) / 16);
      from = reinterpret_cast<const v4u*>(a.digits + (int64_t)block * 16 * a.units * kUnitBytes);
      in_block = min(16, a.M - block * 16);
      row = min(r16, in_block - 1);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int n = 0; n < 4; ++n) d[p][n] = from[digit_at(unit, p, n, row, quad, in_block)];
  };
  v4u digit[2][2][4];
  const auto use = [&](const Unit<NT, GS, S>& c, int unit, int next, int parity) {
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      v4u(&d)[2][4] = digit[SRC == kRead ? (parity + m) & 1 : 0];
      const int row = min(16 * m + r16, rows - 1);
      float worth;
      if constexpr (SRC == kRead) {
        worth = a.worths[(int64_t)(block0 * 16 + row) * a.units + unit];
        if (m + 1 < MB)
          get(unit, m + 1, digit[(parity + m + 1) & 1]);
        else
          get(min(next, a.units - 1), 0, digit[(parity + m + 1) & 1]);
      } else {
        worth = worths[row * a.units + unit];
        get(unit, m, d);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int g = 0; g < 4 / GS; ++g) {
          v4i sum[4];
#pragma unroll
          for (int n = 0; n < 4; ++n) sum[n] = v4i{0, 0, 0, 0};
          if constexpr (GS == 1) {
            const v2u w = {even(c.code[t][g]), odd(c.code[t][g])};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const v2u z = {d[g / 2][n][2 * (g % 2)], d[g / 2][n][2 * (g % 2) + 1]};
              sum[n] = __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, w),
                                                             __builtin_bit_cast(long, z), sum[n], 0, 0, 0);
            }
          } else {
#pragma unroll
            for (int p = g * GS / 2; p < (g + 1) * GS / 2; ++p) {
              const uint32_t c0 = c.code[t][2 * p], c1 = c.code[t][2 * p + 1];
              const v4u w = {even(c0), odd(c0), even(c1), odd(c1)};
#pragma unroll
              for (int n = 0; n < 4; ++n)
                sum[n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, w),
                                                               __builtin_bit_cast(v4i, d[p][n]), sum[n], 0, 0, 0);
            }
          }
          // |sum| <= 128 * 128 * 128: two digits' fit a word
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float lo = (float)(sum[0][i] + sum[1][i] * 256), hi = (float)(sum[2][i] + sum[3][i] * 256);
            acc[t][m][i] = __builtin_fmaf(__builtin_fmaf(hi, 65536.0f, lo) * (float)c.scale[t][g][i], worth, acc[t][m][i]);
          }
        }
        // A tile's sums are joined here: the compiler would put that off past the next loads'
        // branches, with all tiles' sums in registers until then.
        asm volatile("" : "+v"(acc[t][m]));
      }
    }
  };
  if (SRC == kRead && first < a.units) get(first, 0, digit[0]);
  for (int u = first; u < a.units; u += 2 * step) {
    use(x, u, u + step, 0);
    if (u + step >= a.units) break;
    if (u + 2 * step < a.units) x.fetch(a, tile0, u + 2 * step, lane);
    use(y, u + step, u + 2 * step, MB & 1);
    if (u + 3 * step < a.units) y.fetch(a, tile0, u + 3 * step, lane);
  }

  // the waves' sums: box[wave][row][channel of the workgroup's]
  if constexpr (SRC != kRead) __syncthreads();
  float* const box = reinterpret_cast<float*>(smem);
  constexpr int kCh = NT * 16, kOne = MB * 16 * kCh;
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
      *reinterpret_cast<v4f*>(box + wave * kOne + (16 * m + r16) * kCh + 16 * t + 4 * quad) = acc[t][m];
  __syncthreads();
  for (int i = tid; i < rows * kCh; i += kThreads) {
    const int r = i / kCh, n = blockIdx.x * kCh + i % kCh;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += box[w * kOne + i];
    if (n >= a.N) continue;
    if (a.splits > 1)
      a.part[((int64_t)blockIdx.z * a.M + block0 * 16 + r) * a.N + n] = v;
    else
      a.Y[(int64_t)(block0 * 16 + r) * a.ldy + n] = a.bias ? v + a.bias[n] : v;
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

// How a call is cut. Digits are formed in every workgroup while that is little work (up
// to 16384 values; at 2 x 1152 a launch of its own for them makes 11 us of 7), else once.
// More than 16 rows go to workgroups by 16, by 32 or 48 where those still fill 200 compute
// units (77 rows, K 4608, N 1151: 22 us by 48, 18 by 32, 20 by 16).
//
// A workgroup takes 1, 2, 4 or 6 tiles, whichever ends first where workgroups run in rounds of
// one a compute unit and a round takes the time of its tiles and of about one more (its digits and
// its joining; two and a half where digits of groups of 64 or 128 come from memory). 8 rows, K 4096,
// groups of 64, bf16 scales, us by 1, 2, 4 and 6 tiles:
//   N 12288 19.6 19.2 16.7 20.0    N 16400 27.8 25.2 26.9 20.6    N 24576 37.3 28.7 30.7 24.7
//   N 24592 41.0 34.8 30.7 36.7    N 28672 42.5 35.9 31.6 38.4    N 49152 69.1 51.3 44.9 42.6
// 2 rows of fp32, K 1152, N 16400: 9.3 9.8 11.8 8.9; 16 rows, K 4096, N 18432, digits from memory:
// 36.1 29.9 27.1 21.3. Fewer tiles where a unit's scales leave too few registers (N 24576, K 4096):
// fp32 scales in groups of 32 take two at most (44 36 46 75; bf16 ones all six, 44 36 38 32), and
// digits from memory four, in groups of 32 (48 37 40 40) and with fp32 scales in groups of 64 (45 33
// 30 34). Two tiles of 48 rows in groups of 32 spill up to 37 registers and still pay (48 rows: 95
// us, one tile 109; 77 rows, N 4608: 54, 51).
struct Cut {
  int src, NT, MB, splits;
};
// The most tiles of a workgroup for its form.
constexpr int most_tiles(int src, int group, bool s_bf16) {
  return group == 32 ? (!s_bf16 ? 2 : src == kRead ? 4 : 6)
                     : group == 64 && src == kRead && !s_bf16 ? 4 : 6;
}
Cut cut(int M, int N, int K, int group, bool s_bf16) {
  Cut c{};
  const int tiles = (N + 15) / 16, units = (K + kUnit - 1) / kUnit;
  c.MB = M > 32 && tiles * (int64_t)((M + 47) / 48) >= 200 ? 3 : M > 16 && tiles * (int64_t)((M + 31) / 32) >= 200 ? 2 : 1;
  const int64_t groups = (M + 16 * c.MB - 1) / (16 * c.MB);
  const bool fits = M <= 16 && digit_bytes(M, units) + M * units * 4 <= kXBytes;
  c.src = !fits ? kRead : M * units * kUnit <= 16384 ? kForm : kCopy;
  const int most = c.MB > 1 ? 2 : most_tiles(c.src, group, s_bf16);
  const int more = c.src == kRead && group > 32 ? 5 : 2;  // of half tiles
  int64_t best = 0;
  for (const int n : {1, 2, 4, 6}) {
    const int64_t rounds = ((tiles + n - 1) / n * groups + 255) / 256, time = rounds * (2 * n + more);
    if (n <= most && (n == 1 || time <= best)) {
      best = time;
      c.NT = n;
    }
  }
  const int64_t base = (tiles + c.NT - 1) / c.NT * groups;
  int64_t n = 256 / base;
  if (base > 96 || units < 16) n = 1;
  if (n > units / 8) n = units / 8;
  c.splits = (int)(n < 1 ? 1 : n > 16 ? 16 : n);
  return c;
}

template <int NT, int MB, int GS, int SRC, typename S>
hipError_t run(const Rows4Args& a, hipStream_t s) {
  if constexpr (SRC != kForm)
    k_rows4_digits<<<dim3((a.units + 15) / 16, a.M < 32768 ? a.M : 32768, (a.M + 32767) / 32768), 256, 0, s>>>(a);
  const int x = SRC == kRead ? 0 : digit_bytes(a.M, a.units) + a.M * a.units * 4;
  constexpr int box = kWaves * NT * MB * 1024;
  static_assert(box <= kXBytes, "kXBytes is the most that a call asks for");
  const int lds = x > box ? x : box;
  if (lds > 64 * 1024) {
    const hipError_t e = allow_lds<&k_rows4<NT, MB, GS, SRC, S>, kXBytes>();
    if (e != hipSuccess) return e;
  }
  const int blocks = (a.M + 15) / 16;
  const dim3 grid((a.tiles + NT - 1) / NT, (blocks + MB - 1) / MB, a.splits);
  k_rows4<NT, MB, GS, SRC, S><<<grid, kThreads, lds, s>>>(a);
  return hipGetLastError();
}

template <int NT, int MB, int SRC, typename S>
hipError_t pick_group(const Rows4Args& a, hipStream_t s) {
  constexpr bool b = sizeof(S) == 2;
  if constexpr (MB > 1 || NT <= most_tiles(SRC, 32, b))
    if (a.group == 32) return run<NT, MB, 1, SRC, S>(a, s);
  if constexpr (MB > 1 || NT <= most_tiles(SRC, 64, b))
    if (a.group == 64) return run<NT, MB, 2, SRC, S>(a, s);
  return a.group == 128 ? run<NT, MB, 4, SRC, S>(a, s) : hipErrorInvalidValue;
}

template <int NT, int MB, int SRC>
hipError_t pick(const Rows4Args& a, hipStream_t s) {
  return a.s_bf16 ? pick_group<NT, MB, SRC, bf16>(a, s) : pick_group<NT, MB, SRC, float>(a, s);
}

// ------------------------------------------------------------------ layout ----

struct PackArgs {
  const int8_t* codes;    // [N, K]
  const void* scales;     // [N, groups]
  const void* W;          // quantize: [N, K]
  uint32_t* packed;
  void* packed_scales;
  int N, K, units, tiles, groups, group, spots;  // spots: groups with those past K
  bool s_bf16, w_bf16;
};

__device__ __forceinline__ float w_at(const PackArgs& a, int64_t i) {
  return a.w_bf16 ? (float)reinterpret_cast<const bf16*>(a.W)[i]
                  : reinterpret_cast<const float*>(a.W)[i];
}

// Word of channel n's inputs 8 (k / 8) .. + 7.
__device__ __forceinline__ int64_t word_at(const PackArgs& a, int n, int k) {
  return (((int64_t)(n / 16) * a.units + k / 128) * 64 + 16 * (k % 32 / 8) + n % 16) * 4 + k % 128 / 32;
}

// One word a thread.
__global__ __launch_bounds__(256) void k_rows4_pack(PackArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.tiles * a.units * 256) return;
  const int step = (int)(i % 4), lane = (int)(i / 4 % 64), unit = (int)(i / 256 % a.units);
  const int n = (int)(i / 256 / a.units) * 16 + lane % 16, k = unit * 128 + step * 32 + 8 * (lane / 16);
  uint32_t w = 0;
  if (n < a.N && k < a.K)  // K is a multiple of 16
    for (int j = 0; j < 8; ++j)
      w |= ((uint32_t)a.codes[(int64_t)n * a.K + k + j] & 15u) << (4 * j);
  a.packed[i] = w;
}

// One scale a thread; in packed order.
__global__ __launch_bounds__(256) void k_rows4_pack_scales(PackArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.tiles * a.spots * 16) return;
  const int r = (int)(i % 16), g = (int)(i / 16 % a.spots), n = (int)(i / 16 / a.spots) * 16 + r;
  const bool in = n < a.N && g < a.groups;
  const int64_t at = (int64_t)n * a.groups + g;
  if (a.s_bf16)
    reinterpret_cast<bf16*>(a.packed_scales)[i] =
        in ? reinterpret_cast<const bf16*>(a.scales)[at] : (bf16)0.0f;
  else
    reinterpret_cast<float*>(a.packed_scales)[i] =
        in ? reinterpret_cast<const float*>(a.scales)[at] : 0.0f;
}

// One group of one channel a thread: its scale, then its codes by that scale.
__global__ __launch_bounds__(256) void k_rows4_quantize(PackArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.tiles * a.spots * 16) return;
  const int r = (int)(i % 16), g = (int)(i / 16 % a.spots), tile = (int)(i / 16 / a.spots);
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
  for (int k = k0; k < k0 + a.group; k += 8) {
    uint32_t w = 0;
    for (int j = 0; j < 8; ++j) {
      int c = 0;
      if (n < a.N && k + j < a.K && s > 0.0f)
        c = (int)fminf(fmaxf(rintf(w_at(a, (int64_t)n * a.K + k + j) / s), -7.0f), 7.0f);
      w |= ((uint32_t)c & 15u) << (4 * j);
    }
    a.packed[word_at(a, n, k)] = w;
  }
}

// Eight codes or one scale a thread: a launch has less than 2^32 of them.
__global__ __launch_bounds__(256) void k_rows4_unpack(PackArgs a, int8_t* codes, void* scales) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (codes && i < (int64_t)a.N * (a.K / 8)) {
    const int n = (int)(i / (a.K / 8)), k = (int)(i % (a.K / 8)) * 8;
    const uint32_t w = a.packed[word_at(a, n, k)];
    for (int j = 0; j < 8; ++j)
      codes[(int64_t)n * a.K + k + j] = (int8_t)((int)(w << (28 - 4 * j)) >> 28);
  }
  if (scales && i < (int64_t)a.N * a.groups) {
    const int n = (int)(i / a.groups), g = (int)(i % a.groups);
    const int64_t at = ((int64_t)(n / 16) * a.spots + g) * 16 + n % 16;
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
  a.units = l.units;
  a.spots = l.spots;
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
  l.units = (d.K + kUnit - 1) / kUnit;
  l.groups = (d.K + d.group - 1) / d.group;
  l.spots = l.units * (kUnit / d.group);
  l.scales = (int64_t)l.tiles * l.units * 1024;
  l.bytes = l.scales + (int64_t)l.tiles * l.spots * 16 * (d.s_dtype == QL_BF16 ? 2 : 4);
  return l;
}

Rows4Ws rows4_ws(const ql_rows4& d, int M) {
  Rows4Ws w{};
  if (M < 1) return w;
  const Cut c = cut(M, d.N, d.K, d.group, d.s_dtype == QL_BF16);
  const int64_t units = (d.K + kUnit - 1) / kUnit, blocks = (M + 15) / 16;
  if (c.src != kForm) {
    w.worths = blocks * 16 * units * kUnitBytes;
    w.part = w.worths + (M * units * 4 + 15) / 16 * 16;
  }
  w.bytes = w.part + (c.splits > 1 ? (int64_t)c.splits * M * d.N * 4 : 0);
  return w;
}

hipError_t launch_rows4(const Rows4Args& args, hipStream_t s) {
  Rows4Args a = args;
  const Cut c = cut(a.M, a.N, a.K, a.group, a.s_bf16);
  a.splits = c.splits;
  hipError_t e = hipErrorInvalidValue;
#define QL_ROWS4(T)                                               \
  if (c.MB == 1 && c.NT == T)                                     \
    e = c.src == kForm   ? pick<T, 1, kForm>(a, s)                \
        : c.src == kCopy ? pick<T, 1, kCopy>(a, s)                \
                         : pick<T, 1, kRead>(a, s);
  QL_ROWS4(1)
  QL_ROWS4(2)
  QL_ROWS4(4)
  QL_ROWS4(6)
#undef QL_ROWS4
#define QL_ROWS4(T, B) \
  if (c.NT == T && c.MB == B) e = pick<T, B, kRead>(a, s);
  QL_ROWS4(1, 2)
  QL_ROWS4(2, 2)
  QL_ROWS4(1, 3)
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
  k_rows4_pack<<<blocks((int64_t)a.tiles * a.units * 256), 256, 0, s>>>(a);
  k_rows4_pack_scales<<<blocks((int64_t)a.tiles * a.spots * 16), 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_rows4_quantize(const ql_rows4& d, const void* W, bool w_bf16, void* packed,
                                 hipStream_t s) {
  PackArgs a = pack_args(d, packed);
  a.W = W;
  a.w_bf16 = w_bf16;
  k_rows4_quantize<<<blocks((int64_t)a.tiles * a.spots * 16), 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_rows4_unpack(const ql_rows4& d, int8_t* codes, void* scales, hipStream_t s) {
  const PackArgs a = pack_args(d, d.packed);
  const int64_t n = (int64_t)a.N * (a.K / 8), m = (int64_t)a.N * a.groups;
  k_rows4_unpack<<<blocks(n > m ? n : m), 256, 0, s>>>(a, codes, scales);
  return hipGetLastError();
}

}  // namespace ql
