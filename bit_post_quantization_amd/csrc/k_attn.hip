// Attention of queries to the states of another sequence, forward and backward.
//
//   forward   S = scale Q K^T,  P = softmax(S),  O = P V
//   backward  P = exp(S - lse),  delta = rowsum(dO O),  dS = P (dO V^T - delta),
//             dQ = scale dS K  (k_attn_dq),  dV = P^T dO and dK = scale dS^T Q (k_attn_dkv)
//
// A wave owns 32 rows (queries; in k_attn_dkv 32 keys), one a lane of each half
// wave, and walks over tiles of the other side in LDS. Every product is taken so that
// what the wave owns is the column of the matrix instruction (32x32x16 bf16, or eight
// 32x32x2 fp32): S^T = K Q^T leaves a lane 16 scores of its own query for 32 keys,
//   C[4 h + 8 (i / 4) + i % 4][lane % 32], h = lane / 32, i < 16,
// so row maxima and sums stay in the lane but for one exchange between the halves, and
// the scores, rounded, already are the operand of the next product (O^T += V^T P^T,
// dQ^T += K^T dS^T): its 16 keys of step s are the lane's values 8 s .. 8 s + 7, and V^T is
// read from LDS in that order (ds_read_b64_tr_b16 for bf16, single words for fp32). No
// score goes through LDS, nothing is exchanged between waves until the end.
//
// The softmax runs in base 2 (scale2 = scale log2 e), one pass, with the running
// maximum and sum in fp32; O is rescaled only where a maximum of the wave rose past 2^8.
// Roundings: bf16 tensors give bf16 weights P and, in the gradient, bf16 dS (off by at
// most 2^-8 of themselves, as the rounded result is), which the bf16 instruction takes at 7.7
// times the fp32 one's rate; fp32 tensors stay fp32 throughout.
//
// Measured per call (MI355X; bf16 unless said; the library's bf16 matrix product reaches
// 1185 TFLOP/s here, its fp32 one 154, a copy 5.4 TB/s):
//   2 x 4096 queries, 4608 keys, 16 heads of 128: 337-349 us, 890-920 TFLOP/s (the first calls
//     after a pause take up to 372, before the clock is up)
//   16 x 1024 queries, prompts of up to 120 keys, 16 heads of 72: 24 us, 3.3 TB/s
//   4 x 1 query over 4608 keys, 16 heads of 64: 19 us, 3.9 TB/s
//   gradient, 2 x 8190 queries, prompts of 512 and 156, 16 heads on 8 of 128: 257-277 us,
//     400-430 TFLOP/s of the five products that it takes (seven are done), 680 for two
//     sequences of 4096 x 4096 with 16 heads
//   gradient, 8 x 256 queries, 77 keys with holes, 16 heads of 72, fp32: 66-71 us
//   fp32, 2 x 2048 queries and keys: 8 heads of 128 287 us, 16 of 72 371, gradient of 16 of 72
//     1437; 4 x 1 query over 4608 keys, 16 heads of 64: 52
// What bounds the large ones: the way of operands from LDS. It is latency, not LDS's rate (busy 34 %
// of the first case, 24-26 % of the gradient, without conflicts): the products of two waves a SIMD
// do not cover it (with operands from registers instead the first case takes 239 us). 64 rows a wave,
// which would halve the reads, do not fit two waves a SIMD at 128 channels, and with one the
// compiler keeps neither file free of copies (438 us). k_attn_dkv, whose tiles are 32 rows with one
// more on its way, waits 58 % of its waves' time; in fp32 it also leaves waves without keys idle.
//
// This file is compiled once for each type and number DC of 16-channel blocks
// of a head (QL_AT_T, QL_AT_DC); heads of other sizes are padded with zeros in LDS.
#include "ql_block.h"
#include "ql_device.h"

namespace ql {

namespace {

typedef __bf16 bf16;
typedef float f32;
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v8f __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef bf16 v8h __attribute__((ext_vector_type(8)));
typedef bf16 v4h __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s* lds_v4s;

#define QL_AT_F32_f32 1
#define QL_AT_F32_bf16 0
#define QL_AT_IS_F32_(t) QL_AT_F32_##t
#define QL_AT_IS_F32(t) QL_AT_IS_F32_(t)
// Few keys stay in LDS (k_attn_short, attn_plan): all but long heads.
#define QL_AT_SHORT (QL_AT_IS_F32(QL_AT_T) ? QL_AT_DC <= 6 : QL_AT_DC <= 8)

typedef QL_AT_T T;
constexpr int DC = QL_AT_DC;
constexpr int kChunk = 16 / sizeof(T);        // elements of a 16-byte piece
constexpr int kD = 16 * DC;                   // padded channels
constexpr int kOB = (DC + 1) / 2;             // 32-channel blocks of a result
constexpr int kCPR = kD / kChunk;             // pieces of a padded row
constexpr int kThreads = 256;

// Eight elements of one row: an operand's part of a lane.
template <typename E> struct Frag;
template <> struct Frag<bf16> { typedef v8h t; };
template <> struct Frag<f32> { typedef v8f t; };
typedef Frag<T>::t frag;

template <typename V>
__device__ __forceinline__ v16f mma(const V& a, const V& b, v16f c) {
  if constexpr (sizeof(V) == 16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
}

// Values 8 s .. 8 s + 7 of a result as an operand of the next product.
__device__ __forceinline__ frag operand(const v16f& c, int s) {
  frag f;
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = (T)c[8 * s + e];
  return f;
}

// A tile's rows in LDS are read both ways: whole rows by neighbouring lanes, 16 bytes each
// (sixteen lanes meet all 64 banks once), and, for bf16, four rows by 32 channels
// transposed. Both are free of conflicts, without padding, if the 16-byte piece c of row r
// lies at c ^ turn(r). Rows are kOB times 64 bytes: an odd number of them spreads four rows
// over all banks, and turn() needs four values for the rows four apart; rows of 128 bytes
// alternate between two halves, and need eight; rows of 256 all start alike, and need
// sixteen. (Rows padded to an odd number of pieces cost the gradients 45 % of their LDS
// time.) fp32 rows, whose columns are read by words, are an odd number of pieces long.
constexpr bool kTurned = sizeof(T) == 2;
constexpr int kPitch = kTurned ? kOB * 32 : ((kOB * 32 / kChunk) | 1) * kChunk;
static_assert(kOB <= 5, "turn() for longer rows");
constexpr int kTurn = kOB == 4 ? 128 : kOB == 2 ? 64 : 32;  // elements that trade places
__device__ __forceinline__ int turn(int r) {
  return (kOB == 4 ? (r & 3) << 2 : kOB == 2 ? (r & 2) << 1 : 0) | ((r >> 2) & 3);
}
__device__ __forceinline__ int place(int r, int c) {
  return r * kPitch + (kTurned ? (c ^ turn(r)) : c) * kChunk;
}
// From the place of a row's first channels to that of the channels `by` further on, a
// multiple of 16.
__device__ __forceinline__ constexpr int further(int at, int by) {
  return (at ^ (by & (kTurn - 1))) + (by & ~(kTurn - 1));
}

// A lane's places in a tile.
struct Spots {
  int row, col;
  __device__ __forceinline__ void find(int lane) {
    const int r32 = lane & 31, h = lane >> 5, i = lane & 15;
    if constexpr (kTurned) {
      row = place(r32, h);
      col = place(4 * h + i / 4, 2 * ((lane >> 4) & 1) + ((i & 3) >> 1)) + 4 * (i & 1);
    } else {
      row = r32 * kPitch + 8 * h;
      col = 4 * h * kPitch + r32;
    }
  }
};

// The places of a tile's operands are formed from two registers for each tile: kept over the
// loop they would take sixteen, and spill.
__device__ __forceinline__ void form_anew(Spots& s) { asm volatile("" : "+v"(s.row), "+v"(s.col)); }

// Operand of rows: row lane % 32 of p, channels 16 kb + 8 h .. + 7.
template <typename E>
__device__ __forceinline__ typename Frag<E>::t row_frag(const E* p, const Spots& s, int kb) {
  if constexpr (sizeof(E) == 2)
    return *reinterpret_cast<const v8h*>(p + further(s.row, 16 * kb));
  else
    return *reinterpret_cast<const v8f*>(p + s.row + 16 * kb);
}

// Operand of columns: channel 32 c + lane % 32, rows 4 h .. + 3 and 8 + 4 h .. + 3 of p.
template <typename E>
__device__ __forceinline__ typename Frag<E>::t col_frag(const E* p, const Spots& s, int c) {
  if constexpr (sizeof(E) == 2) {
    // eight rows on, turn() differs by 2: 16 channels
    const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p + further(s.col, 32 * c)));
    const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_v4s)(p + further(s.col ^ 16, 32 * c) + 8 * kPitch));
    return __builtin_bit_cast(v8h, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
  } else {
    const E* a = p + s.col + 32 * c;
    v8f f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = a[e * kPitch];
      f[4 + e] = a[(8 + e) * kPitch];
    }
    return f;
  }
}

__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32); }
__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

constexpr float kSlack = 8.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Workgroup `id` of B Hk runs of `per` (the tiles of one key head) in an order that keeps
// `a.unit` neighbouring heads' runs in one L2: workgroups are dealt to the 8 XCDs in turn.
// Neighbouring units go to unlike XCDs where they divide evenly.
__device__ __forceinline__ int by_xcd(const AttnArgs& a, int id, int per) {
  const int x = id % 8, j = id / 8, n = a.B * a.Hk * per;
  per *= a.unit;
  if (n / per % 8 == 0) return (j / per * 8 + x) * per + j % per;
  return x * (n / 8) + min(x, n % 8) + j;
}

__device__ __forceinline__ void split_row(const AttnArgs& a, int r, int& l, int& g) {
  l = a.G == 1 ? r : r / a.G;
  g = a.G == 1 ? 0 : r - l * a.G;
}

__device__ __forceinline__ const T* row_of(const AttnArgs& a, const ql_heads_view& t, int b, int hk,
                                           int r) {
  int l, g;
  split_row(a, r, l, g);
  return reinterpret_cast<const T*>(t.p) + b * t.batch + l * t.row + (int64_t)(hk * a.G + g) * t.head;
}

// Place of row r in a [B, H, Lq] array.
__device__ __forceinline__ int64_t stat_at(const AttnArgs& a, int b, int hk, int r) {
  int l, g;
  split_row(a, r, l, g);
  return ((int64_t)b * a.H + hk * a.G + g) * a.Lq + l;
}

// Eight channels of a row in memory, zero past D.
__device__ __forceinline__ frag load_frag(const T* row, int c, int D) {
  frag f;
  if (c < D) {
    f = *reinterpret_cast<const frag*>(row + c);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (T)0.0f;
  }
  return f;
}

// The rows of a wave as operands, by way of LDS: neighbouring lanes load neighbouring
// pieces of a row, which the load path takes four at a time, where the operand's own order,
// a row a lane, goes piece by piece (two thirds of k_attn_dq's time for q, dO and O). `room`
// is the wave's own, 32 kPitch elements.
struct Rows {
  static constexpr int N = (32 * kCPR + 63) / 64;
  v4u r[N];
  template <typename F>
  __device__ __forceinline__ void fetch(int lane, int D, F address) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = lane + 64 * i;
      r[i] = *reinterpret_cast<const v4u*>(address(min(at / kCPR, 31)) +
                                           min(at % kCPR, D / kChunk - 1) * kChunk);
    }
  }
  __device__ __forceinline__ void operands(T* room, const Spots& s, int lane, int D,
                                           frag (&out)[DC]) const {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = lane + 64 * i;
      v4u x = r[i];
      if (D < kD && at % kCPR * kChunk >= D) x = v4u{0, 0, 0, 0};
      if (32 * kCPR % 64 == 0 || at < 32 * kCPR)
        *reinterpret_cast<v4u*>(room + place(at / kCPR, at % kCPR)) = x;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int kb = 0; kb < DC; ++kb) out[kb] = row_frag(room, s, kb);
  }
};

// A row of a result, times f, to memory. A lane has four channels in eight; in bf16 the
// halves of the wave trade two such pieces, so that each stores eight in one piece.
template <typename E>
__device__ __forceinline__ void store_row(E* p, const v16f (&c)[kOB], float f, int D, int h) {
#pragma unroll
  for (int i = 0; i < kOB; ++i) {
    if constexpr (sizeof(E) == 2) {
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        v4h x, y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = (E)(c[i][4 * j + e] * f);
          y[e] = (E)(c[i][4 * j + 4 + e] * f);
        }
        const v2u u = __builtin_bit_cast(v2u, x), v = __builtin_bit_cast(v2u, y);
        const auto lo = __builtin_amdgcn_permlane32_swap(u[0], v[0], false, false);
        const auto hi = __builtin_amdgcn_permlane32_swap(u[1], v[1], false, false);
        const int d = 32 * i + 8 * j + 8 * h;
        if (d < D) *reinterpret_cast<v4u*>(p + d) = v4u{lo[0], hi[0], lo[1], hi[1]};
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = 32 * i + 8 * j + 4 * h;
        v4f o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = c[i][4 * j + e] * f;
        if (d < D) *reinterpret_cast<v4f*>(p + d) = o;
      }
    }
  }
}

__device__ __forceinline__ v16f zero16() {
  v16f z;
#pragma unroll
  for (int e = 0; e < 16; ++e) z[e] = 0.0f;
  return z;
}

// Which of the keys of a tile of 32 W count: a bit each, the same in all lanes.
template <int W>
struct KeyBits {
  uint32_t w[W];
  __device__ __forceinline__ void look(const AttnArgs& a, int b, int key0, int len, int lane) {
    if (!a.mask && key0 + 32 * W <= len) {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = 0xffffffffu;
      return;
    }
#pragma unroll
    for (int i = 0; i < W; i += 2) {
      const int key = key0 + 32 * i + lane;
      bool ok = key < len;
      if (a.mask && ok) ok = a.mask[b * a.mask_batch + key] != 0;
      const uint64_t m = __ballot(ok);
      w[i] = (uint32_t)m;
      if (i + 1 < W) w[i + 1] = (uint32_t)(m >> 32);
    }
  }
  __device__ __forceinline__ bool all() const {
    uint32_t x = w[0];
#pragma unroll
    for (int i = 1; i < W; ++i) x &= w[i];
    return x == 0xffffffffu;
  }
  __device__ __forceinline__ bool none() const {
    uint32_t x = w[0];
#pragma unroll
    for (int i = 1; i < W; ++i) x |= w[i];
    return x == 0;
  }
};

__device__ __forceinline__ int key_len(const AttnArgs& a, int b) {
  if (!a.lens) return a.Lk;
  const int n = a.lens[b];
  return n < 0 ? 0 : n > a.Lk ? a.Lk : n;
}

// The sum of a row that has none, in all lanes of a wave alike: 0 where no key of the sequence
// counts (its result is 0), NaN where keys count and all score -infinity (they have no
// softmax). Looked up only where a row ends so; the loop over the tiles keeps no count.
__device__ __forceinline__ float sum_of_none(const AttnArgs& a, int b, int len, int lane) {
  if (!a.mask) return len > 0 ? NAN : 0.0f;
  for (int key0 = 0; key0 < len; key0 += 64)
    if (__any(key0 + lane < len && a.mask[b * a.mask_batch + key0 + lane] != 0)) return NAN;
  return 0.0f;
}

// A tile of KT rows of one tensor on its way from memory through registers to LDS. Where
// rows lie evenly (row i of a tile, i = u G + g, at u steps and g heads from the tile's
// start) and near, a piece's address is the tile's, which is the same for all lanes, and
// an offset formed once; else it is formed for each tile.
template <int KT>
struct Stage {
  static constexpr int N = (KT * kCPR + kThreads - 1) / kThreads;
  static constexpr bool kWhole = KT * kCPR % kThreads == 0;
  v4u r[N];
  uint32_t off[N];
  int to[N];
  static __device__ __forceinline__ int row(int tid, int i) { return min((tid + i * kThreads) / kCPR, KT - 1); }
  static __device__ __forceinline__ int piece(int tid, int i, int D) {
    return min((tid + i * kThreads) % kCPR, D / kChunk - 1);
  }
  __device__ __forceinline__ void find(int tid, int D, int G, int64_t step, int64_t head) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = row(tid, i), u = G == 1 ? at : at / G, g = G == 1 ? 0 : at - u * G;
      off[i] = (uint32_t)(u * step + g * head) * (uint32_t)sizeof(T) + 16 * piece(tid, i, D);
      to[i] = place(at, (tid + i * kThreads) % kCPR);
    }
  }
  __device__ __forceinline__ void fetch(const T* tile) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      r[i] = *reinterpret_cast<const v4u*>(reinterpret_cast<const char*>(tile) + off[i]);
  }
  // row(i): the address of row i of the tile (any valid one past the end)
  template <typename F>
  __device__ __forceinline__ void fetch_by(int tid, int D, F address) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      r[i] = *reinterpret_cast<const v4u*>(address(row(tid, i)) + piece(tid, i, D) * kChunk);
  }
  // keep(i): whether row i of the tile is kept (else zero); channels past D are zero
  template <bool ALL, typename F>
  __device__ __forceinline__ void put(T* lds, int tid, int D, F keep) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v4u x = r[i];
      if (D < kD && (tid + i * kThreads) % kCPR * kChunk >= D) x = v4u{0, 0, 0, 0};
      if constexpr (!ALL) {
        if (!keep(row(tid, i))) x = v4u{0, 0, 0, 0};
      }
      if (kWhole || tid + i * kThreads < KT * kCPR) *reinterpret_cast<v4u*>(lds + to[i]) = x;
    }
  }
};

template <int W>
__device__ __forceinline__ bool bit_of(const KeyBits<W>& k, int i) {
  uint32_t x = k.w[0];
#pragma unroll
  for (int j = 1; j < W; ++j) x = (i >> 5) == j ? k.w[j] : x;
  return (x >> (i & 31)) & 1;
}

// Waves a SIMD that the registers are to allow: two where they fit, at most eleven of them
// spilled (us with one and with two; bf16, forward, 128 channels: 709, 390, 4 x 4096 queries
// and keys, 8 heads of 160, nine spilled: 545, 371; fp32, 2 x 2048 queries and keys: forward, 8
// heads of 96: 250, 224, 8 of 128: 326, 286 (with tiles of 32 keys, below), but one query a
// sequence and 4096 keys, 16 heads on 8 of 128: 103, 118; gradient, 16 heads of 64: 1112, 920,
// both kernels 8 of 96: 801, 906, 8 of 128: 1036, 1632). Of 160 channels in fp32 LDS holds
// one workgroup, and k_attn_dkv's 32 keys a wave spill 92 registers even so.
constexpr bool kPairs = sizeof(T) == 2;
template <int WK> constexpr int kForwardWaves = kPairs || DC <= (WK == 1 ? 8 : 6) ? 2 : 1;
constexpr int kDqWaves = DC <= (kPairs ? 8 : 6) ? 2 : 1, kDkvWaves = DC <= (kPairs ? 8 : 4) ? 2 : 1;
// Keys of a tile of k_attn_dq; 32 leave long fp32 heads the registers that they need (the
// gradient of 2 x 2048 queries and keys, us: 16 heads of 72: 1472 with 64, 1436 with 32, 8 of
// 96: 795, 782, 8 of 128: 1026, 1039; 8 x 256 queries of 77 keys, 16 heads of 128: 99, 97, of
// 160: 151, 141).
constexpr int kDqKeys = kPairs || DC <= 4 ? 64 : 32;

// ----------------------------------------------------------------- forward ----

// SUB pieces of 32 keys for a wave's rows: scores, the running maximum m and sum l, and
// O += weights times values. words: the keys of each piece that count.
template <int SUB>
__device__ __forceinline__ void attend(const T* kt, const T* vt, const Spots& spots, float scale2,
                                       const uint32_t (&words)[SUB], const frag (&q)[DC],
                                       v16f (&o)[kOB], float& m, float& l, int h) {
  v16f s[SUB];
  uint32_t every = 0xffffffffu;
#pragma unroll
  for (int u = 0; u < SUB; ++u) {
    s[u] = zero16();
    every &= words[u];
#pragma unroll
    for (int kb = 0; kb < DC; ++kb) s[u] = mma(row_frag(kt + 32 * u * kPitch, spots, kb), q[kb], s[u]);
  }
  if (every != 0xffffffffu) {
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      const uint32_t w = words[u] >> (4 * h);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (!((w >> (8 * (i / 4) + i % 4)) & 1)) s[u][i] = -INFINITY;
    }
  }
  float top = s[0][0];
#pragma unroll
  for (int u = 0; u < SUB; ++u)
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, s[u][i]);
  // Weights stay within 2^8 of what the true maximum would make them: O and l are only
  // rescaled where one rose further (the first of them starts from -infinity).
  const float m_new = fmaxf(m, fmaxf(top, other_half(top)) * scale2);
  if (__any(m_new > m + kSlack)) {
    const float f = exp2_fast(m - (m_new == -INFINITY ? 0.0f : m_new));
    l *= f;
#pragma unroll
    for (int i = 0; i < kOB; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[i][e] *= f;
    m = m_new;
  }
  const float base = m == -INFINITY ? 0.0f : m;
  float sum = 0.0f;
#pragma unroll
  for (int u = 0; u < SUB; ++u) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[u][i] = exp2_fast(__builtin_fmaf(s[u][i], scale2, -base));
      sum += s[u][i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const frag p = operand(s[u], i);
      const T* v0 = vt + (32 * u + 16 * i) * kPitch;
#pragma unroll
      for (int c = 0; c < kOB; ++c) o[c] = mma(col_frag(v0, spots, c), p, o[c]);
    }
  }
  l += sum;
}

// O and lse of a row, l being the whole sum (0 only where no key counts).
__device__ __forceinline__ void finish(const AttnArgs& a, int b, int hk, int row, const v16f (&o)[kOB],
                                       float m, float l, int h) {
  const bool empty = l == 0.0f;
  const float inv = empty ? 0.0f : 1.0f / l;
  if (a.lse && h == 0)
    a.lse[stat_at(a, b, hk, row)] = empty ? -INFINITY : (m + __log2f(l)) * kLn2;
  T* p = const_cast<T*>(row_of(a, a.o, b, hk, row));
  store_row(p, o, inv, a.D, h);
}

// Few keys (a prompt's): all of them stay in LDS while a workgroup goes through `per_group`
// tiles of rows, its waves on their own after the one barrier, the next rows' queries under
// way.
#if QL_AT_SHORT
__global__ __launch_bounds__(kThreads, (kForwardWaves<1>)) void k_attn_short(AttnArgs a) {
  constexpr int KT = 64, kTile = KT * 2 * kPitch;
  constexpr bool kRoom = (2 * kTile + 128 * kPitch) * sizeof(T) <= 81920;  // for two workgroups
  __shared__ __attribute__((aligned(16))) T lds[2 * kTile + (kRoom ? 128 * kPitch : 0)];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r32 = lane & 31, h = lane >> 5;
  Spots spots;
  spots.find(lane);
  const int groups = (a.row_tiles + a.per_group - 1) / a.per_group;
  int id = by_xcd(a, blockIdx.x, groups);
  const int rt0 = id % groups * a.per_group, rt1 = min(rt0 + a.per_group, a.row_tiles);
  id /= groups;
  const int hk = id % a.Hk, b = id / a.Hk;
  const int len = key_len(a, b), tiles = (len + KT - 1) / KT;
  const T* const kp = reinterpret_cast<const T*>(a.k.p) + b * a.k.batch + hk * a.k.head;
  const T* const vp = reinterpret_cast<const T*>(a.v.p) + b * a.v.batch + hk * a.v.head;
  frag next[kRoom ? 1 : DC];
  Rows rows;
  const auto ask = [&](int rt) {
    const int r0 = rt * 128 + wave * 32;
    if constexpr (kRoom) {
      rows.fetch(lane, a.D, [&](int i) { return row_of(a, a.q, b, hk, min(r0 + i, a.R - 1)); });
    } else {
      const T* p = row_of(a, a.q, b, hk, min(r0 + r32, a.R - 1));
#pragma unroll
      for (int kb = 0; kb < DC; ++kb) next[kb] = load_frag(p, 16 * kb + 8 * h, a.D);
    }
  };
  ask(rt0);
  KeyBits<2> bits[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    bits[t].look(a, b, t * KT, len, lane);
    if (t < tiles) {
      Stage<KT> ks, vs;
      ks.find(tid, a.D, 1, 0, 0);
      vs.find(tid, a.D, 1, 0, 0);
      ks.fetch_by(tid, a.D, [&](int i) { return kp + (int64_t)min(t * KT + i, a.Lk - 1) * a.k.row; });
      vs.fetch_by(tid, a.D, [&](int i) { return vp + (int64_t)min(t * KT + i, a.Lk - 1) * a.v.row; });
      const auto keep = [&](int i) { return bit_of(bits[t], i); };
      ks.template put<true>(lds + t * kTile, tid, a.D, keep);
      vs.template put<false>(lds + t * kTile + KT * kPitch, tid, a.D, keep);
    }
  }
  __syncthreads();
  for (int rt = rt0; rt < rt1; ++rt) {
    frag q[DC];
    if constexpr (kRoom) {
      rows.operands(lds + 2 * kTile + wave * 32 * kPitch, spots, lane, a.D, q);
    } else {
#pragma unroll
      for (int kb = 0; kb < DC; ++kb) q[kb] = next[kb];
    }
    if (rt + 1 < rt1) ask(rt + 1);
    v16f o[kOB];
#pragma unroll
    for (int i = 0; i < kOB; ++i) o[i] = zero16();
    float m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      form_anew(spots);
      const T* const kt = lds + t * kTile;
      if (bits[t].w[1])
        attend<2>(kt, kt + KT * kPitch, spots, a.scale2, bits[t].w, q, o, m, l, h);
      else if (bits[t].w[0])
        attend<1>(kt, kt + KT * kPitch, spots, a.scale2, {bits[t].w[0]}, q, o, m, l, h);
    }
    const int row = rt * 128 + wave * 32 + r32;
    l += other_half(l);
    if (l == 0.0f && !(bits[0].none() && bits[1].none())) l = NAN;  // as sum_of_none
    if (row < a.R) finish(a, b, hk, row, o, m, l, h);
  }
}
#endif

// WK waves of a workgroup share its keys, 4 / WK its rows: one, or two in fp32 for up to 64
// rows (one query a sequence, us with two and with one: 4 x 4608 keys, 16 heads of 64: 52, 55; 4 x
// 1000 keys 21, 28; 2 x 4096, 8 of 128 38, 47; 64 queries, 2 x 2048 keys, 16 of 72: 29, 37; only of
// many long heads one is faster: 8 x 4096 keys, 16 on 8 of 128: 103, 87). In bf16 few rows
// too are faster with one, the other waves helping to load (8 x 1 query of 32 heads on 8 of
// 128, 4096 keys: 36 us; with four, 57): two tiles fit LDS.
template <int WK>
struct Fwd {
  static constexpr int WQ = 4 / WK, kRows = 32 * WQ;
  // 32-key pieces of a wave in a tile. Long fp32 heads take one, whose way to LDS leaves the
  // registers for a second wave (8 heads of 128: 326 us with two, 286 with one; of 160: 428,
  // 403; of 96 no less with one).
  static constexpr int SUB = WK == 1 && (kPairs || DC <= 6) ? 2 : 1;
  static constexpr int KT = 32 * WK * SUB;
  static constexpr int kTile = KT * 2 * kPitch;
  // Tiles in LDS: two where two workgroups still fit (fp32, 2 x 2048 queries and keys, 16 heads
  // of 72: 419 us with two, 373 with one; bf16, 8 of 160: 83 and 85).
  static constexpr int NB = KT == 32 || (WK == 1 && 4 * kTile * (int)sizeof(T) <= 160 * 1024) ? 2 : 1;
  static constexpr int kJoin = WK > 1 ? (WK - 1) * WQ * 32 * (kOB * 32 + 2) * 4 : 0;
  static constexpr int kLds = NB * kTile * (int)sizeof(T) > kJoin ? NB * kTile * (int)sizeof(T)
                                                                 : kJoin;
  // Where the 128 rows of the waves pass: behind the first tile, or over it.
  static constexpr int kRowsAt = NB * kTile - 128 * kPitch;
  static_assert(kRowsAt >= 0, "the waves' rows fit the tiles");
};

template <int WK>
__global__ __launch_bounds__(kThreads, kForwardWaves<WK>) void k_attn_forward(AttnArgs a) {
  typedef Fwd<WK> P;
  constexpr int KT = P::KT, SUB = P::SUB, W = KT / 32;
  __shared__ __attribute__((aligned(16))) char smem[P::kLds];
  T* const lds = reinterpret_cast<T*>(smem);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wq = wave / WK, wk = wave % WK, r32 = lane & 31, h = lane >> 5;
  int id = by_xcd(a, blockIdx.x, a.row_tiles * a.splits);
  const int sp = id % a.splits;
  id /= a.splits;
  const int rt = id % a.row_tiles;
  id /= a.row_tiles;
  const int hk = id % a.Hk, b = id / a.Hk;
  const int len = key_len(a, b);
  const int tiles = (len + KT - 1) / KT, per = (tiles + a.splits - 1) / a.splits;
  const int t0 = sp * per, t1 = min(tiles, t0 + per);
  const int row0 = rt * P::kRows + wq * 32, row = row0 + r32;
  const bool busy = row0 < a.R;  // else this wave only helps to fill the tiles
  Spots spots;
  spots.find(lane);
  frag q[DC];
  {
    Rows rows;
    rows.fetch(lane, a.D, [&](int i) { return row_of(a, a.q, b, hk, min(row0 + i, a.R - 1)); });
    rows.operands(lds + P::kRowsAt + wave * 32 * kPitch, spots, lane, a.D, q);
    if (P::kRowsAt < P::kTile) __syncthreads();  // the first tile goes there
  }
  const T* const kp = reinterpret_cast<const T*>(a.k.p) + b * a.k.batch + hk * a.k.head;
  const T* const vp = reinterpret_cast<const T*>(a.v.p) + b * a.v.batch + hk * a.v.head;
  v16f o[kOB];
#pragma unroll
  for (int i = 0; i < kOB; ++i) o[i] = zero16();
  float m = -INFINITY, l = 0.0f;

  Stage<KT> ks, vs;
  ks.find(tid, a.D, 1, a.k.row, 0);
  vs.find(tid, a.D, 1, a.v.row, 0);
  KeyBits<W> bits, next;
  const auto fetch = [&](int t) {
    if (a.near_keys && (t + 1) * KT <= a.Lk) {
      ks.fetch(kp + (int64_t)t * KT * a.k.row);
      vs.fetch(vp + (int64_t)t * KT * a.v.row);
    } else {
      ks.fetch_by(tid, a.D, [&](int i) { return kp + (int64_t)min(t * KT + i, a.Lk - 1) * a.k.row; });
      vs.fetch_by(tid, a.D, [&](int i) { return vp + (int64_t)min(t * KT + i, a.Lk - 1) * a.v.row; });
    }
    next.look(a, b, t * KT, len, lane);
  };
  const auto put = [&](T* at) {
    const auto keep = [&](int i) { return bit_of(next, i); };
    ks.template put<true>(at, tid, a.D, keep);  // scores of other keys are not looked at
    if (next.all())
      vs.template put<true>(at + KT * kPitch, tid, a.D, keep);
    else
      vs.template put<false>(at + KT * kPitch, tid, a.D, keep);
  };
  if (t0 < t1) {
    fetch(t0);
    put(lds);
  }
  bits = next;
  __syncthreads();
  for (int t = t0; t < t1; ++t) {
    const T* const kt = lds + ((t - t0) % P::NB) * P::kTile;
    const T* const vt = kt + KT * kPitch;
    if (t + 1 < t1) fetch(t + 1);
    form_anew(spots);
    if (busy && !bits.none()) {
      uint32_t words[SUB];
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        words[u] = 0;  // wk is uniform: a select of the words
#pragma unroll
        for (int j = 0; j < W; ++j) words[u] = j == wk * SUB + u ? bits.w[j] : words[u];
      }
      const int at = wk * SUB * 32 * kPitch;
      attend<SUB>(kt + at, vt + at, spots, a.scale2, words, q, o, m, l, h);
    }
    if constexpr (P::NB == 1) __syncthreads();
    if (t + 1 < t1) put(lds + ((t + 1 - t0) % P::NB) * P::kTile);
    bits = next;
    __syncthreads();
  }
  l += other_half(l);

  if constexpr (WK > 1) {  // the waves of other keys hand over what they have
    float* const box = reinterpret_cast<float*>(smem);
    constexpr int kLd = kOB * 32 + 2;
    if (wk > 0) {
      float* p = box + ((wk - 1) * P::WQ + wq) * 32 * kLd + r32 * kLd;
#pragma unroll
      for (int c = 0; c < kOB; ++c)
#pragma unroll
        for (int e = 0; e < 16; ++e) p[32 * c + 8 * (e / 4) + 4 * h + e % 4] = o[c][e];
      if (h == 0) {
        p[kOB * 32] = m;
        p[kOB * 32 + 1] = l;
      }
    }
    __syncthreads();
    if (wk > 0) return;
    float top = m;
#pragma unroll
    for (int j = 0; j < WK - 1; ++j)
      top = fmaxf(top, box[((j * P::WQ + wq) * 32 + r32) * kLd + kOB * 32]);
    const float base = top == -INFINITY ? 0.0f : top;
    const float f = exp2_fast(m - base);
    l *= f;
#pragma unroll
    for (int c = 0; c < kOB; ++c)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[c][e] *= f;
#pragma unroll
    for (int j = 0; j < WK - 1; ++j) {
      const float* p = box + ((j * P::WQ + wq) * 32 + r32) * kLd;
      const float g = exp2_fast(p[kOB * 32] - base);
      l = __builtin_fmaf(g, p[kOB * 32 + 1], l);
#pragma unroll
      for (int c = 0; c < kOB; ++c)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          o[c][e] = __builtin_fmaf(g, p[32 * c + 8 * (e / 4) + 4 * h + e % 4], o[c][e]);
    }
    m = top;
  }
  if (a.splits == 1 && __any(l == 0.0f)) {
    const float none = sum_of_none(a, b, len, lane);
    l = l == 0.0f ? none : l;
  }
  if (row >= a.R) return;
  if (a.splits == 1) return finish(a, b, hk, row, o, m, l, h);
  const bool empty = l == 0.0f;  // k_attn_join looks whether any part has keys
  const float inv = empty ? 0.0f : 1.0f / l;
  const int64_t n = (int64_t)a.B * a.H * a.Lq, at = stat_at(a, b, hk, row);
  float* p = a.part + (sp * n + at) * a.D;
  if (h == 0) a.part_lse[sp * n + at] = empty ? -INFINITY : m + __log2f(l);
  store_row(p, o, inv, a.D, h);
}

// One wave a row: the parts of its splits weighted by their share of the sum. Lane s
// has split s's share; the parts' loads wait for nothing.
__global__ __launch_bounds__(kThreads) void k_attn_join(AttnArgs a) {
  const int64_t n = (int64_t)a.B * a.H * a.Lq;
  const int64_t at = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (at >= n) return;
  const int lane = threadIdx.x & 63;
  const float mine = lane < a.splits ? a.part_lse[lane * n + at] : -INFINITY;  // splits <= 64
  float acc[3] = {0.0f, 0.0f, 0.0f}, top = mine;
  for (int i = 1; i < 64; i *= 2) top = fmaxf(top, __shfl_xor(top, i));
  const float share = exp2_fast(mine - (top == -INFINITY ? 0.0f : top));
  float total = share;
  for (int i = 1; i < 64; i *= 2) total += __shfl_xor(total, i);
  for (int s0 = 0; s0 < a.splits; s0 += 8) {
    float p[8][3];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float* from = a.part + (min(s0 + j, a.splits - 1) * n + at) * a.D;
#pragma unroll
      for (int i = 0; i < 3; ++i) p[j][i] = lane + 64 * i < a.D ? from[lane + 64 * i] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = s0 + j < a.splits ? __shfl(share, s0 + j) : 0.0f;
#pragma unroll
      for (int i = 0; i < 3; ++i) acc[i] = __builtin_fmaf(f, p[j][i], acc[i]);
    }
  }
  const int l = (int)(at % a.Lq);
  const int64_t bh = at / a.Lq;
  if (total == 0.0f) total = sum_of_none(a, (int)(bh / a.H), key_len(a, (int)(bh / a.H)), lane);
  const bool empty = total == 0.0f;
  const float inv = empty ? 0.0f : 1.0f / total;
  T* p = reinterpret_cast<T*>(a.o.p) + bh / a.H * a.o.batch + l * a.o.row + bh % a.H * a.o.head;
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (lane + 64 * i < a.D) p[lane + 64 * i] = (T)(acc[i] * inv);
  if (a.lse && lane == 0) a.lse[at] = empty ? -INFINITY : (top + __log2f(total)) * kLn2;
}

// ---------------------------------------------------------------- backward ----

constexpr int kBackRows = 32;  // rows of a tile in LDS of k_attn_dkv
constexpr bool kKeepV = sizeof(T) == 2 && DC >= 8;

// dQ, and delta for k_attn_dkv. Keys that do not count are zero in LDS and have P = 0.
__global__ __launch_bounds__(kThreads, kDqWaves) void k_attn_dq(AttnArgs a) {
  constexpr int KT = kDqKeys, W = KT / 32, kTile = KT * 2 * kPitch;
  constexpr int NB = KT == 32 || 2 * kTile * (int)sizeof(T) <= 81920 ? 2 : 1;
  constexpr int kRowsAt = NB * kTile - 128 * kPitch;  // where the 128 rows of the waves pass
  static_assert(kRowsAt >= 0, "the waves' rows fit the tiles");
  __shared__ __attribute__((aligned(16))) T lds[NB * kTile];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r32 = lane & 31, h = lane >> 5;
  int id = by_xcd(a, blockIdx.x, a.row_tiles);
  const int rt = id % a.row_tiles;
  id /= a.row_tiles;
  const int hk = id % a.Hk, b = id / a.Hk;
  const int len = key_len(a, b), tiles = (len + KT - 1) / KT;
  const int row0 = rt * 128 + wave * 32, row = row0 + r32;
  const bool busy = row0 < a.R;  // else this wave only helps to fill the tiles
  const int64_t at = stat_at(a, b, hk, min(row, a.R - 1));
  Spots spots;
  spots.find(lane);

  frag q[DC], g[DC];
  float delta = 0.0f;
  {
    T* const room = lds + kRowsAt + wave * 32 * kPitch;
    Rows rq, rg, ro;
    rq.fetch(lane, a.D, [&](int i) { return row_of(a, a.q, b, hk, min(row0 + i, a.R - 1)); });
    rg.fetch(lane, a.D, [&](int i) { return row_of(a, a.dout, b, hk, min(row0 + i, a.R - 1)); });
    ro.fetch(lane, a.D, [&](int i) { return row_of(a, a.o, b, hk, min(row0 + i, a.R - 1)); });
    frag o[DC];
    rq.operands(room, spots, lane, a.D, q);
    rg.operands(room, spots, lane, a.D, g);
    ro.operands(room, spots, lane, a.D, o);
#pragma unroll
    for (int kb = 0; kb < DC; ++kb)
#pragma unroll
      for (int e = 0; e < 8; ++e) delta = __builtin_fmaf((float)g[kb][e], (float)o[kb][e], delta);
    delta += other_half(delta);
    if (h == 0 && row < a.R) a.delta[at] = delta;
    if (kRowsAt < kTile) __syncthreads();  // the first tile goes there
  }
  // back in base two: one rounding more, of P's own size times 2^-24 |lse|, as the saved lse's own
  float lse2 = a.lse[at] * kLog2e;
  if (lse2 == -INFINITY) lse2 = INFINITY;  // no key counts: P = 0
  const T* const kp = reinterpret_cast<const T*>(a.k.p) + b * a.k.batch + hk * a.k.head;
  const T* const vp = reinterpret_cast<const T*>(a.v.p) + b * a.v.batch + hk * a.v.head;
  v16f dq[kOB];
#pragma unroll
  for (int i = 0; i < kOB; ++i) dq[i] = zero16();

  Stage<KT> ks, vs;
  ks.find(tid, a.D, 1, a.k.row, 0);
  vs.find(tid, a.D, 1, a.v.row, 0);
  KeyBits<W> bits, next;
  const auto fetch = [&](int t) {
    if (a.near_keys && (t + 1) * KT <= a.Lk) {
      ks.fetch(kp + (int64_t)t * KT * a.k.row);
      vs.fetch(vp + (int64_t)t * KT * a.v.row);
    } else {
      ks.fetch_by(tid, a.D, [&](int i) { return kp + (int64_t)min(t * KT + i, a.Lk - 1) * a.k.row; });
      vs.fetch_by(tid, a.D, [&](int i) { return vp + (int64_t)min(t * KT + i, a.Lk - 1) * a.v.row; });
    }
    next.look(a, b, t * KT, len, lane);
  };
  const auto put = [&](T* to) {
    const auto keep = [&](int i) { return bit_of(next, i); };
    if (next.all()) {
      ks.template put<true>(to, tid, a.D, keep);
      vs.template put<true>(to + KT * kPitch, tid, a.D, keep);
    } else {
      ks.template put<false>(to, tid, a.D, keep);
      vs.template put<false>(to + KT * kPitch, tid, a.D, keep);
    }
  };
  if (tiles > 0) {
    fetch(0);
    put(lds);
  }
  bits = next;
  __syncthreads();
  for (int t = 0; t < tiles; ++t) {
    const T* const kt = lds + (t % NB) * kTile;
    const T* const vt = kt + KT * kPitch;
    if (t + 1 < tiles) fetch(t + 1);
    form_anew(spots);
    if (busy && !bits.none()) {
#pragma unroll
      for (int u = 0; u < W; ++u) {
        if (!bits.w[u]) continue;
        v16f s = zero16(), dp = zero16();
#pragma unroll
        for (int kb = 0; kb < DC; ++kb) {
          s = mma(row_frag(kt + 32 * u * kPitch, spots, kb), q[kb], s);
          dp = mma(row_frag(vt + 32 * u * kPitch, spots, kb), g[kb], dp);
        }
        const uint32_t w = bits.w[u] >> (4 * h);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float p = exp2_fast(__builtin_fmaf(s[i], a.scale2, -lse2));
          s[i] = p * (dp[i] - delta);
        }
        if (bits.w[u] != 0xffffffffu) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (!((w >> (8 * (i / 4) + i % 4)) & 1)) s[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const frag ds = operand(s, i);
          const T* k0 = kt + (32 * u + 16 * i) * kPitch;
#pragma unroll
          for (int c = 0; c < kOB; ++c) dq[c] = mma(col_frag(k0, spots, c), ds, dq[c]);
        }
      }
    }
    if constexpr (NB == 1) __syncthreads();
    if (t + 1 < tiles) put(lds + ((t + 1) % NB) * kTile);
    bits = next;
    __syncthreads();
  }
  if (row >= a.R) return;
  T* p = const_cast<T*>(row_of(a, a.dq, b, hk, row));
  store_row(p, dq, a.scale, a.D, h);
}

// Where tiles of keys are shared out (a.splits > 1, at most 256 sequences), the workgroups
// of a key head, B key_tiles splits of them, are dealt to the tiles that have a key
// that counts, all sequences together and all tiles alike: sequences differ in length, and
// a tile's rows should not wait while others' workgroups have nothing to do.
struct Deal {
  int share;          // workgroups of a tile; 0: there is no such tile
  int b, tile, turn;  // workgroup w's: sequence, tile of its keys, which of the sharers
};
constexpr int kMostShared = 256;
__device__ __forceinline__ int used_tiles(const AttnArgs& a, int b) {
  return b < a.B ? (key_len(a, b) + 127) / 128 : 0;
}
__device__ __forceinline__ Deal deal(const AttnArgs& a, int w, int lane) {
  constexpr int N = kMostShared / 64;
  int used[N], upto[N], total = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    used[i] = used_tiles(a, 64 * i + lane);
    int n = used[i];
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int o = __shfl_up(n, d);
      if (lane >= d) n += o;
    }
    upto[i] = total + n;
    total += __builtin_amdgcn_readlane(n, 63);
  }
  Deal out = {total ? a.B * a.key_tiles * a.splits / total : 0, 0, 0, 0};
  if (!out.share) return out;
  const int t = w / out.share;
  if (t >= total) return Deal{0, 0, 0, 0};  // what does not divide evenly
  out.turn = w - t * out.share;
#pragma unroll
  for (int i = N - 1; i >= 0; --i) {
    const uint64_t past = __ballot(upto[i] > t);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      out.b = 64 * i + l;
      out.tile = t - (__builtin_amdgcn_readlane(upto[i], l) - __builtin_amdgcn_readlane(used[i], l));
    }
  }
  return out;
}

// dK and dV of 128 keys from a range of the rows; a lane has one key. With long heads V
// stays in LDS, so that the registers leave room for two waves a SIMD.
__global__ __launch_bounds__(kThreads, kDkvWaves) void k_attn_dkv(AttnArgs a) {
  constexpr int RT = kBackRows, kTile = RT * 2 * kPitch;
  constexpr int NB = 2;
  __shared__ __attribute__((aligned(16))) T lds[NB * kTile];
  __shared__ __attribute__((aligned(16))) float stats[NB][2][RT];
  __shared__ __attribute__((aligned(16))) T v_rows[kKeepV ? 128 * kPitch : 8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r32 = lane & 31, h = lane >> 5;
  T* const my_v = v_rows + (kKeepV ? wave * 32 * kPitch : 0);
  int b, hk, kt, sp, share, place_of;
  if (a.splits == 1) {
    place_of = by_xcd(a, blockIdx.x, a.key_tiles);
    kt = place_of % a.key_tiles;
    hk = place_of / a.key_tiles % a.Hk;
    b = place_of / a.key_tiles / a.Hk;
    sp = 0;
    share = 1;
  } else {  // heads in runs, so that those whose number 8 divides keep to one L2
    const int all = a.B * a.key_tiles * a.splits;
    place_of = a.Hk % 8 == 0 ? (blockIdx.x / 8 / all * 8 + blockIdx.x % 8) * all + blockIdx.x / 8 % all
                             : blockIdx.x;
    hk = place_of / all;
    const Deal d = deal(a, place_of % all, lane);
    if (!d.share) return;
    b = d.b;
    kt = d.tile;
    sp = d.turn;
    share = d.share;
  }
  const int len = key_len(a, b), key = kt * 128 + wave * 32 + r32;
  bool counts = key < len;
  if (a.mask && counts) counts = a.mask[b * a.mask_batch + key] != 0;
  const bool busy = __any(counts);  // else this wave only helps to fill the tiles
  const int tiles = (a.R + RT - 1) / RT, per = (tiles + share - 1) / share;
  const int t0 = sp * per, t1 = kt * 128 < len ? min(tiles, t0 + per) : 0;

  Spots spots;
  spots.find(lane);
  frag k[DC], v[kKeepV ? 1 : DC];
  {
    const int key0 = kt * 128 + wave * 32;
    T* const room = kKeepV ? my_v : lds + wave * (NB * kTile / 4);
    const T* const kp = reinterpret_cast<const T*>(a.k.p) + b * a.k.batch + hk * a.k.head;
    const T* const vp = reinterpret_cast<const T*>(a.v.p) + b * a.v.batch + hk * a.v.head;
    Rows rk, rv;
    rk.fetch(lane, a.D, [&](int i) { return kp + (int64_t)min(key0 + i, a.Lk - 1) * a.k.row; });
    rv.fetch(lane, a.D, [&](int i) { return vp + (int64_t)min(key0 + i, a.Lk - 1) * a.v.row; });
    rk.operands(room, spots, lane, a.D, k);
    frag x[DC];
    rv.operands(room, spots, lane, a.D, x);  // my_v: where V stays
    if constexpr (!kKeepV) {
#pragma unroll
      for (int kb = 0; kb < DC; ++kb) v[kKeepV ? 0 : kb] = x[kb];
      __syncthreads();
    }
  }
  v16f dk[kOB], dv[kOB];
#pragma unroll
  for (int i = 0; i < kOB; ++i) dk[i] = dv[i] = zero16();

  Stage<RT> qs, gs;
  qs.find(tid, a.D, a.G, a.q.row, a.q.head);
  gs.find(tid, a.D, a.G, a.dout.row, a.dout.head);
  float stat = 0.0f;  // of thread t < RT lse of row t, of t < 2 RT delta of row t - RT
  const auto fetch = [&](int t) {
    if (a.near_rows && (t + 1) * RT <= a.R) {
      qs.fetch(row_of(a, a.q, b, hk, t * RT));
      gs.fetch(row_of(a, a.dout, b, hk, t * RT));
    } else {
      qs.fetch_by(tid, a.D, [&](int i) { return row_of(a, a.q, b, hk, min(t * RT + i, a.R - 1)); });
      gs.fetch_by(tid, a.D, [&](int i) { return row_of(a, a.dout, b, hk, min(t * RT + i, a.R - 1)); });
    }
    if (tid < 2 * RT) {
      const int r = t * RT + tid % RT;
      const int64_t at = stat_at(a, b, hk, min(r, a.R - 1));
      if (tid < RT) {
        stat = a.lse[at] * kLog2e;  // rounded as in k_attn_dq
        if (stat == -INFINITY || r >= a.R) stat = INFINITY;  // P = 0
      } else {
        stat = r < a.R ? a.delta[at] : 0.0f;
      }
    }
  };
  const auto put = [&](int t) {
    const int n = a.R - t * RT, at = (t - t0) % NB;
    T* to = lds + at * kTile;
    const auto keep = [&](int i) { return i < n; };
    // Past the last row dO is zero and q that row again: with an lse of infinity P is 0 there
    // whenever the last row's own is a number, also for a key of -infinity, where q = 0
    // would score NaN.
    qs.template put<true>(to, tid, a.D, keep);
    if (n >= RT)
      gs.template put<true>(to + RT * kPitch, tid, a.D, keep);
    else
      gs.template put<false>(to + RT * kPitch, tid, a.D, keep);
    if (tid < 2 * RT) stats[at][tid / RT][tid % RT] = stat;
  };
  if (t0 < t1) {
    fetch(t0);
    put(t0);
  }
  __syncthreads();
  for (int t = t0; t < t1; ++t) {
    const int at = (t - t0) % NB;
    const T* const qt = lds + at * kTile;
    const T* const gt = qt + RT * kPitch;
    if (t + 1 < t1) fetch(t + 1);
    form_anew(spots);
    if (busy) {
    v16f s = zero16(), dp = zero16();
#pragma unroll
    for (int kb = 0; kb < DC; ++kb) {
      s = mma(row_frag(qt, spots, kb), k[kb], s);
      dp = mma(row_frag(gt, spots, kb), kKeepV ? row_frag(my_v, spots, kb) : v[kKeepV ? 0 : kb], dp);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const v4f lse2 = *reinterpret_cast<const v4f*>(&stats[at][0][8 * j + 4 * h]);
      const v4f delta = *reinterpret_cast<const v4f*>(&stats[at][1][8 * j + 4 * h]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = exp2_fast(__builtin_fmaf(s[4 * j + e], a.scale2, -lse2[e]));
        s[4 * j + e] = p;
        dp[4 * j + e] = p * (dp[4 * j + e] - delta[e]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const frag p = operand(s, i), ds = operand(dp, i);
#pragma unroll
      for (int c = 0; c < kOB; ++c) {
        dv[c] = mma(col_frag(gt + 16 * i * kPitch, spots, c), p, dv[c]);
        dk[c] = mma(col_frag(qt + 16 * i * kPitch, spots, c), ds, dk[c]);
      }
    }
    }
    if (t + 1 < t1) put(t + 1);
    __syncthreads();
  }
  if (key >= a.Lk || (a.splits > 1 && !counts)) return;  // k_attn_dkv_sum knows them too
  if (!counts) {  // whatever their columns hold
#pragma unroll
    for (int i = 0; i < kOB; ++i) dk[i] = dv[i] = zero16();
  }
  if (a.splits > 1) {
    float* p = a.part + ((int64_t)place_of * 256 + key % 128) * a.D;
    store_row(p, dk, a.scale, a.D, h);
    store_row(p + 128 * a.D, dv, 1.0f, a.D, h);
    return;
  }
  T* pk = reinterpret_cast<T*>(a.dk.p) + b * a.dk.batch + key * a.dk.row + hk * a.dk.head;
  T* pv = reinterpret_cast<T*>(a.dv.p) + b * a.dv.batch + key * a.dv.row + hk * a.dv.head;
  store_row(pk, dk, a.scale, a.D, h);
  store_row(pv, dv, 1.0f, a.D, h);
}

// dK (blockIdx.y 0) and dV (1): the sum of the row ranges' parts, four channels a thread.
__global__ __launch_bounds__(kThreads) void k_attn_dkv_sum(AttnArgs a) {
  __shared__ int before[kMostShared + 1];  // tiles with keys that count of the sequences before
  const int lane = threadIdx.x & 63;
  if (threadIdx.x < 64) {
    int base = 0;
#pragma unroll
    for (int i = 0; i < kMostShared / 64; ++i) {
      int n = used_tiles(a, 64 * i + lane);
      const int mine = n;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(n, d);
        if (lane >= d) n += o;
      }
      before[64 * i + lane] = base + n - mine;
      base += __builtin_amdgcn_readlane(n, 63);
    }
    if (lane == 0) before[kMostShared] = base;
  }
  __syncthreads();
  const int64_t n = (int64_t)a.B * a.Lk * a.Hk * a.D;
  const int64_t e = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
  if (e >= n) return;
  const ql_heads_view& t = blockIdx.y ? a.dv : a.dk;
  const int64_t row = e / a.D, lh = row / a.Hk;
  const int b = (int)(lh / a.Lk), key = (int)(lh - (int64_t)b * a.Lk), len = key_len(a, b);
  const int all = a.B * a.key_tiles * a.splits, total = before[kMostShared];
  const int share = total ? all / total : 0;
  const int64_t first = row % a.Hk * all + (int64_t)(before[b] + key / 128) * share;
  const float* p = a.part + (first * 256 + blockIdx.y * 128 + key % 128) * a.D + e % a.D;
  bool counts = key < len;
  if (a.mask && counts) counts = a.mask[b * a.mask_batch + key] != 0;
  v4f sum = {0, 0, 0, 0};
  if (counts) {
    for (int s0 = 0; s0 < share; s0 += 8) {
      v4f x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        x[j] = *reinterpret_cast<const v4f*>(p + min(s0 + j, share - 1) * 256 * (int64_t)a.D);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (s0 + j < share) sum += x[j];
    }
  }
  T* to = reinterpret_cast<T*>(t.p) + lh / a.Lk * t.batch + lh % a.Lk * t.row + row % a.Hk * t.head +
          e % a.D;
  if constexpr (sizeof(T) == 2) {
    v4h o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (T)sum[i];
    *reinterpret_cast<v4h*>(to) = o;
  } else {
    *reinterpret_cast<v4f*>(to) = sum;
  }
}

}  // namespace

#define QL_CAT3(a, b, c, d) a##b##c##d
#define QL_NAME(f, t, d) QL_CAT3(f, t, _, d)

hipError_t QL_NAME(attn_forward_, QL_AT_T, QL_AT_DC)(const AttnArgs& a, const AttnPlan& p,
                                                     hipStream_t s) {
  const int grid = a.B * a.Hk * a.row_tiles * a.splits;
#if QL_AT_SHORT
  if (p.per_group > 0) {
    const int groups = (a.row_tiles + a.per_group - 1) / a.per_group;
    k_attn_short<<<a.B * a.Hk * groups, kThreads, 0, s>>>(a);
    return hipGetLastError();
  }
#endif
  if (sizeof(T) == 4 && p.narrow)
    k_attn_forward<sizeof(T) == 4 ? 2 : 1><<<grid, kThreads, 0, s>>>(a);
  else
    k_attn_forward<1><<<grid, kThreads, 0, s>>>(a);
  if (a.splits > 1) {
    const int64_t n = (int64_t)a.B * a.H * a.Lq;
    k_attn_join<<<(int)((n + 3) / 4), kThreads, 0, s>>>(a);
  }
  return hipGetLastError();
}

hipError_t QL_NAME(attn_grad_, QL_AT_T, QL_AT_DC)(const AttnArgs& args, const AttnPlan& p,
                                                  hipStream_t s) {
  AttnArgs a = args;
  a.row_tiles = p.q_tiles;
  a.key_tiles = p.key_tiles;
  a.splits = p.k_splits;
  if (a.R > 0) k_attn_dq<<<a.B * a.Hk * a.row_tiles, kThreads, 0, s>>>(a);
  if (a.Lk > 0) {
    k_attn_dkv<<<a.B * a.Hk * a.key_tiles * a.splits, kThreads, 0, s>>>(a);
    if (a.splits > 1) {
      const int64_t n = (int64_t)a.B * a.Lk * a.Hk * a.D;
      k_attn_dkv_sum<<<dim3((int)((n / 4 + kThreads - 1) / kThreads), 2), kThreads, 0, s>>>(a);
    }
  }
  return hipGetLastError();
}

}  // namespace ql
