// Low-rank adapters of many requests beside one shared projection.
//
//   forward   S = X A_a^T,  Y = base + scale_a S B_a^T
//             small outputs: k_lora_forward; large ones: k_lora_s, k_lora_expand
//   backward  dS = scale_a dY B_a and dB_a = scale_a dY^T S    (k_lora_grad_y)
//             dX = dS A_a and dA_a = dS^T X                    (k_lora_grad_x)
//             dA, dB summed over the row ranges                (k_lora_slot_sum)
//
// All of it is bound by memory: a rank of 64 makes 2 r = 128 operations an element
// of base that is read and written, far below what the matrix cores do in that
// time. So what the kernels are built for is one reading of every large operand,
// loads that run ahead, and addresses in an order that memory likes.
//
// A tile of rows never spans two requests, so it has one adapter; each workgroup
// finds its tile from the request offsets by one scan over them. Sums are fp32, with
// no atomics and in a fixed order, so a call gives the same bits every time.
//
// Products: where both operands are bf16, v_mfma_f32_16x16x32_bf16. An fp32 operand
// beside a bf16 one is split into three bf16 terms (v = h + m + l holds fp32's 24 bits),
// also where the result is rounded to bf16: sums that cancel show every bit. Where
// both are fp32, v_mfma_f32_16x16x4_f32, or both split where the sums run over rows.
//
// Measured per call (MI355X; what a copy of the same bytes would take in brackets):
//   8 rows, K 1152, N 6912, rank 16, bf16, 8 adapters: 6.5 us of kernel, 7.6 us a call
//   1003 rows of 23 requests, N 1001, rank 12: 12.0 us
//   guided 4096 rows, K 1152, N 4608, rank 16, fp32: 24.6 us (17)
//   16384 rows, K 2048, N 8192, rank 64, bf16: 239 us, 4.8 TB/s (212)
//   gradients of 2048 rows, K 1152, N 4608, rank 16, fp32: 36 us (11)
//   gradients of 16384 rows, K 4608, N 1152, rank 64, bf16: 173 us (72)
#include "ql_device.h"
#include "ql_ops.h"

namespace ql {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 bf16;
typedef bf16 v8h __attribute__((ext_vector_type(8)));

// Request and rows of tile t when every request's rows are cut into tiles of
// T. Uniform over the wave; false past the last tile.
struct Tile {
  int row0, rows, adapter;
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// A lane looks at four requests, so that one trip to memory covers 256 of them.
__device__ bool find_tile(const Requests& q, int T, int t, Tile& out) {
  constexpr int kEach = 4;
  const int lane = threadIdx.x & (kWave - 1);
  int done = 0;
  for (int base = 0; base < q.n; base += kEach * kWave) {
    int off[kEach + 1], id[kEach];
#pragma unroll
    for (int k = 0; k <= kEach; ++k) off[k] = q.off[min(base + lane * kEach + k, q.n)];
#pragma unroll
    for (int k = 0; k < kEach; ++k) id[k] = q.ids[min(base + lane * kEach + k, q.n - 1)];
    int begin[kEach], end[kEach], tiles[kEach], sum = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      begin[k] = clampi(off[k], 0, q.rows);
      end[k] = clampi(off[k + 1], begin[k], q.rows);
      tiles[k] = base + lane * kEach + k < q.n ? (end[k] - begin[k] + T - 1) / T : 0;
      sum += tiles[k];
    }
    const int incl = wave_scan(sum, lane);
    const int total = __builtin_amdgcn_readlane(incl, kWave - 1);
    if (t < done + total) {
      const int src = __ffsll((unsigned long long)__ballot(done + incl > t)) - 1;
      int first = done + __builtin_amdgcn_readlane(incl - sum, src);  // tiles before request k
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int nt = __builtin_amdgcn_readlane(tiles[k], src);
        if (t < first + nt) {
          out.row0 = __builtin_amdgcn_readlane(begin[k], src) + (t - first) * T;
          out.rows = min(T, __builtin_amdgcn_readlane(end[k], src) - out.row0);
          const int a = __builtin_amdgcn_readlane(id[k], src);
          out.adapter = a >= 0 && a < q.n_adapters ? a : -1;
          return true;
        }
        first += nt;
      }
    }
    done += total;
  }
  return false;
}

__device__ __forceinline__ int rank_of(const int32_t* ranks, int a, int rank) {
  return ranks ? clampi(ranks[a], 0, rank) : rank;
}

// Four consecutive elements; `valid` of them exist (the rest are zero and not
// read). vec: p is 16-byte aligned.
__device__ __forceinline__ void load_4(const float* p, int valid, bool vec, float (&v)[4]) {
  if (vec && valid >= 4) {
    const v4f x = *reinterpret_cast<const v4f*>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = x[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = e < valid ? p[e] : 0.0f;
  }
}

__device__ __forceinline__ v4f mfma_f32(float a, float b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// ----------------------------------------------------------------- forward ----
// One workgroup: a tile of MT * 16 rows (of both halves when guided) and a
// share of the output columns. First the tile's S = X A^T, the waves taking
// every NW-th chunk of K and joining their sums in LDS; then the waves stream
// 64 columns at a time: base in, base + S B^T out.
//
// With bf16 adapters the second product takes S in three bf16 terms (24 bits: Y is
// fp32): 6 matrix instructions of 16 cycles for 16x16 outputs at rank 64, where the
// fp32 instructions would take 512 cycles.

__device__ __forceinline__ v4f mfma_bf16(v8h a, v8h b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// v = h + m + l with bf16 terms (24 bits together); a non-finite v stays in h.
__device__ __forceinline__ void split3(float v, bf16& h, bf16& m, bf16& l) {
  h = (bf16)v;
  const float r = __builtin_isfinite((float)h) ? v - (float)h : 0.0f;
  m = (bf16)r;
  l = (bf16)(r - (float)m);
}

// One operand of a 32-column step: elements 8 g .. 8 g + 7 of a row.
template <typename T>
struct Frag8;
template <>
struct Frag8<bf16> {
  v8h v;
  __device__ __forceinline__ void load(const bf16* p) { v = *reinterpret_cast<const v8h*>(p); }
  __device__ __forceinline__ void load(const bf16* p, int valid) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < valid ? p[e] : (bf16)0.0f;
  }
  __device__ __forceinline__ float get(int e) const { return (float)v[e]; }
};
template <>
struct Frag8<float> {
  v4f a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const v4f*>(p);
    b = *reinterpret_cast<const v4f*>(p + 4);
  }
  __device__ __forceinline__ void load(const float* p, int valid) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = e < valid ? p[e] : 0.0f;
      b[e] = e + 4 < valid ? p[e + 4] : 0.0f;
    }
  }
  __device__ __forceinline__ float get(int e) const { return e < 4 ? a[e] : b[e - 4]; }
};

// c += a b over 32 columns (the order of the columns within a sum is free).
template <typename TA, typename TB>
__device__ __forceinline__ v4f step32(const Frag8<TA>& a, const Frag8<TB>& b, v4f c) {
  if constexpr (sizeof(TA) == 2 && sizeof(TB) == 2) {
    return mfma_bf16(a.v, b.v, c);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = mfma_f32(a.get(e), b.get(e), c);
    return c;
  }
}

// S fragments of MT row tiles in registers, for products with rows of B.
template <typename WT, int RT, int MT>
struct SFrag;
template <int RT, int MT>
struct SFrag<float, RT, MT> {  // element e: rank 16 r + 4 g + e
  typedef v4f vec;
  vec s[MT][RT];
  __device__ __forceinline__ void load(const float* lds, int ld, int r16, int g) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < RT; ++r)
        s[m][r] = *reinterpret_cast<const v4f*>(lds + (m * 16 + r16) * ld + r * 16 + 4 * g);
  }
};
template <int RT, int MT>
struct SFrag<bf16, RT, MT> {  // element e: rank 32 k + 8 g + e (RT = 1: see below)
  static constexpr int KS = RT == 1 ? 2 : 3 * RT / 2;
  typedef v8h vec;
  vec s[MT][KS];
  __device__ __forceinline__ void load(const float* lds, int ld, int r16, int g) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const float* p = lds + (m * 16 + r16) * ld;
      if constexpr (RT == 1) {  // 16 ranks: terms h and m in one product, l in the other
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          bf16 h, mi, l;
          split3(p[8 * (g & 1) + e], h, mi, l);
          s[m][0][e] = g < 2 ? h : mi;
          s[m][1][e] = g < 2 ? l : (bf16)0.0f;
        }
      } else {
#pragma unroll
        for (int k = 0; k < RT / 2; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            bf16 h, mi, l;
            split3(p[32 * k + 8 * g + e], h, mi, l);
            s[m][3 * k][e] = h;
            s[m][3 * k + 1][e] = mi;
            s[m][3 * k + 2][e] = l;
          }
      }
    }
  }
};

// One row of B (16 RT ranks at most, `ra` of them used), shared by all rows of S.
template <typename WT, int RT>
struct BFrag;
template <int RT>
struct BFrag<float, RT> {
  float b[RT][4];
  __device__ __forceinline__ void load(const float* row, int ra, bool vec, int g) {
#pragma unroll
    for (int r = 0; r < RT; ++r) load_4(row + r * 16 + 4 * g, ra - r * 16 - 4 * g, vec, b[r]);
  }
  // The same from a column of A: element j at p[j * ld].
  __device__ __forceinline__ void load_column(const float* p, int64_t ld, int ra, int g) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = r * 16 + 4 * g + e;
        b[r][e] = j < ra ? p[j * ld] : 0.0f;
      }
  }
  // lane: row 4 g + i of S's tile, the product with this lane's row of B
  template <int MT>
  __device__ __forceinline__ v4f times(const SFrag<float, RT, MT>& s, int m) const {
    v4f c{0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) c = mfma_f32(s.s[m][r][e], b[r][e], c);
    return c;
  }
};
template <int RT>
struct BFrag<bf16, RT> {
  static constexpr int KB = RT == 1 ? 1 : RT / 2;
  v8h b[KB];
  __device__ __forceinline__ void load(const bf16* row, int ra, bool vec, int g) {
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const int j = RT == 1 ? 8 * (g & 1) : 32 * k + 8 * g;
      if (vec && ra - j >= 8) {
        b[k] = *reinterpret_cast<const v8h*>(row + j);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) b[k][e] = j + e < ra ? row[j + e] : (bf16)0.0f;
      }
    }
  }
  __device__ __forceinline__ void load_column(const bf16* p, int64_t ld, int ra, int g) {
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = (RT == 1 ? 8 * (g & 1) : 32 * k + 8 * g) + e;
        b[k][e] = j < ra ? p[j * ld] : (bf16)0.0f;
      }
  }
  template <int MT>
  __device__ __forceinline__ v4f times(const SFrag<bf16, RT, MT>& s, int m) const {
    v4f c{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < SFrag<bf16, RT, MT>::KS; ++k)
      c = mfma_bf16(s.s[m][k], b[RT == 1 ? 0 : k / 3], c);
    return c;
  }
};

// A wave's output block: MT * 16 rows times 64 columns, four products side by
// side. Neighbouring lanes have neighbouring addresses, which the load path
// needs (it takes 64 bytes of neighbouring lanes at a time, else 16: with rows side
// by side in the lanes instead, 16384 x 8192 at rank 64 took 299 us, now 207): with VEC
// product u has columns 4 (lane % 16) + u, so a lane ends up with four columns
// in a row of each of its four rows 4 g + i; without, columns 16 u + lane % 16
// and single elements.
constexpr int kBlockCols = 64;
template <bool VEC>
__device__ __forceinline__ int block_col(int u, int r16) {
  return VEC ? 4 * r16 + u : 16 * u + r16;
}

template <int MT, bool VEC>
struct Block {
  float v[MT][4][4];  // [row tile][row 4 g + i][u]

  __device__ __forceinline__ void load(const float* base, int64_t ld, int row0, int rows, int n0,
                                       int N, int r16, int g) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* p = base + (int64_t)(row0 + min(m * 16 + 4 * g + i, rows - 1)) * ld + n0;
        if (VEC && n0 + 4 * r16 + 4 <= N) {
          const v4f x = *reinterpret_cast<const v4f*>(p + 4 * r16);
#pragma unroll
          for (int u = 0; u < 4; ++u) v[m][i][u] = x[u];
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int c = block_col<VEC>(u, r16);
            v[m][i][u] = n0 + c < N ? p[c] : 0.0f;
          }
        }
      }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) v[m][i][u] = 0.0f;
  }
  template <typename WT, int RT>
  __device__ __forceinline__ void add(const SFrag<WT, RT, MT>& s, const BFrag<WT, RT>& b, int u) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const v4f c = b.times(s, m);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[m][i][u] += c[i];
    }
  }
  __device__ __forceinline__ void store(float* Y, int64_t ld, int row0, int rows, int n0, int N,
                                        int r16, int g) const {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = m * 16 + 4 * g + i;
        if (row >= rows) continue;
        float* p = Y + (int64_t)(row0 + row) * ld + n0;
        if (VEC && n0 + 4 * r16 + 4 <= N) {
          *reinterpret_cast<v4f*>(p + 4 * r16) = v4f{v[m][i][0], v[m][i][1], v[m][i][2], v[m][i][3]};
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int c = block_col<VEC>(u, r16);
            if (n0 + c < N) p[c] = v[m][i][u];
          }
        }
      }
  }
};

template <int RT, int MT, int H, int NW>
struct SBuf {  // partial sums of the waves; [0][row][rank] holds S in the end
  float v[NW][H * MT * 16][RT * 16 + 4];
};

// S = X A^T of one tile by the whole workgroup, combined over the halves and
// scaled, into buf.v[0] (ranks past `ra` and rows of a bare tile are zero). The
// waves take every NW-th chunk of K and join their sums in LDS. With `save`,
// the tile's rows of a.S receive S as it was before the combine and the scale.
template <typename XT, typename WT, int RT, int MT, int H, int NW>
__device__ void tile_s(const ForwardArgs& a, const Tile& t, int ra, float sc, bool xvec, bool save,
                       SBuf<RT, MT, H, NW>& buf) {
  constexpr int T = MT * 16, R = RT * 16;
  constexpr int CH = sizeof(XT) == 2 ? 64 : 32;  // columns of 128 bytes of X
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, g = lane >> 4;
  const bool bare = t.adapter < 0;
  auto& red = buf.v;
  if (!bare) {
    const XT* X = reinterpret_cast<const XT*>(a.X);
    const WT* A = reinterpret_cast<const WT*>(a.A) + (int64_t)t.adapter * a.rank * a.K;
    const XT* xp[H * MT];
    const WT* wp[RT];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int m = 0; m < MT; ++m)
        xp[h * MT + m] = X + (int64_t)(h * a.q.rows + t.row0 + min(m * 16 + r16, t.rows - 1)) * a.ldx +
                         8 * g;
    // rank rows past the stored ones: another row, dropped below
#pragma unroll
    for (int r = 0; r < RT; ++r) wp[r] = A + (int64_t)min(r * 16 + r16, a.rank - 1) * a.K + 8 * g;
    v4f acc[H * MT][RT];
#pragma unroll
    for (int m = 0; m < H * MT; ++m)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[m][r] = v4f{0, 0, 0, 0};
    int c = wave * CH;
    if (xvec && c + CH <= a.K) {  // whole chunks, the next one's loads ahead of this one's products
      Frag8<XT> x[CH / 32][H * MT], nx[CH / 32][H * MT];
      Frag8<WT> w[CH / 32][RT], nw[CH / 32][RT];
      auto load = [&](int at, Frag8<XT>(&fx)[CH / 32][H * MT], Frag8<WT>(&fw)[CH / 32][RT]) {
#pragma unroll
        for (int u = 0; u < CH / 32; ++u) {
#pragma unroll
          for (int m = 0; m < H * MT; ++m) fx[u][m].load(xp[m] + at + 32 * u);
#pragma unroll
          for (int r = 0; r < RT; ++r) fw[u][r].load(wp[r] + at + 32 * u);
        }
      };
      load(c, x, w);
      for (; c + CH <= a.K; c += NW * CH) {
        if (c + NW * CH + CH <= a.K) load(c + NW * CH, nx, nw);
#pragma unroll
        for (int u = 0; u < CH / 32; ++u)
#pragma unroll
          for (int m = 0; m < H * MT; ++m)
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[m][r] = step32(w[u][r], x[u][m], acc[m][r]);
#pragma unroll
        for (int u = 0; u < CH / 32; ++u) {
#pragma unroll
          for (int m = 0; m < H * MT; ++m) x[u][m] = nx[u][m];
#pragma unroll
          for (int r = 0; r < RT; ++r) w[u][r] = nw[u][r];
        }
      }
    }
    for (; c < a.K; c += NW * CH) {  // the last, short chunk, and unaligned X
      for (int k = c; k < min(c + CH, a.K); k += 32) {
        const int valid = k + 8 * g < a.K ? 8 : 0;  // K % 16 == 0
        Frag8<XT> x[H * MT];
        Frag8<WT> w[RT];
#pragma unroll
        for (int m = 0; m < H * MT; ++m) x[m].load(xp[m] + k, valid);
#pragma unroll
        for (int r = 0; r < RT; ++r) w[r].load(wp[r] + k, valid);
#pragma unroll
        for (int m = 0; m < H * MT; ++m)
#pragma unroll
          for (int r = 0; r < RT; ++r) acc[m][r] = step32(w[r], x[m], acc[m][r]);
      }
    }
    // acc[m][r][i]: row 16 m + lane % 16, rank 16 r + 4 g + i
#pragma unroll
    for (int m = 0; m < H * MT; ++m)
#pragma unroll
      for (int r = 0; r < RT; ++r)
        *reinterpret_cast<v4f*>(&red[wave][m * 16 + r16][r * 16 + 4 * g]) = acc[m][r];
  }
  __syncthreads();
  // Sum over the waves, the guided combine, the scale: red[0][row][rank].
  for (int u = threadIdx.x; u < T * R / 4; u += 64 * NW) {
    const int row = u / (R / 4), j = u % (R / 4) * 4;
    v4f s{0, 0, 0, 0};
    if (!bare) {
      s = *reinterpret_cast<v4f*>(&red[0][row][j]);
#pragma unroll
      for (int w = 1; w < NW; ++w) s += *reinterpret_cast<v4f*>(&red[w][row][j]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e >= ra) s[e] = 0.0f;
    if (save && row < t.rows) {
      float* o = a.S + (int64_t)(t.row0 + row) * a.rank + j;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e < a.rank) o[e] = s[e];
    }
    if constexpr (H == 2) {
      v4f n{0, 0, 0, 0};
      if (!bare) {
        n = *reinterpret_cast<v4f*>(&red[0][T + row][j]);
#pragma unroll
        for (int w = 1; w < NW; ++w) n += *reinterpret_cast<v4f*>(&red[w][T + row][j]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e >= ra) n[e] = 0.0f;
      if (save && row < t.rows) {
        float* o = a.S + (int64_t)(a.q.rows + t.row0 + row) * a.rank + j;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < a.rank) o[e] = n[e];
      }
      s = n + a.w * (s - n);
    }
    *reinterpret_cast<v4f*>(&red[0][row][j]) = s * sc;
  }
  __syncthreads();
}

// All in one: right for calls so small that a second launch costs more than
// computing S again in the workgroups that share a tile. What bounds it is latency:
// about four trips to memory one after another (offsets, X and A, base and B, Y),
// 6.4 us for 8 rows, most of the host's time for the call.
template <typename XT, typename WT, int RT, int MT, int H, int NW, bool YVEC>
__global__ __launch_bounds__(64 * NW) void k_lora_forward(ForwardArgs a, bool xvec, bool bvec) {
  constexpr int T = MT * 16, LD = RT * 16 + 4;
  __shared__ __align__(16) SBuf<RT, MT, H, NW> buf;
  // Workgroups of one tile follow each other on one chiplet (workgroup ids go
  // round the eight of them), so that they find the tile's X in its L2.
  const int xcd = blockIdx.x & 7, loc = blockIdx.x >> 3;
  const int tile = loc / a.shares * 8 + xcd, share = loc % a.shares;
  Tile t;
  if (!find_tile(a.q, T, tile, t)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, g = lane >> 4;
  const bool bare = t.adapter < 0;
  if (bare && a.base == a.Y && !a.S) return;
  const int ra = bare ? 0 : rank_of(a.ranks, t.adapter, a.rank);
  const float sc = bare ? 0.0f : a.scales ? a.scales[t.adapter] : 1.0f;
  tile_s<XT, WT, RT, MT, H, NW>(a, t, ra, sc, xvec, a.S && share == 0, buf);
  if (bare && a.base == a.Y) return;
  SFrag<WT, RT, MT> sf;
  if (!bare) sf.load(&buf.v[0][0][0], LD, r16, g);
  const WT* B = reinterpret_cast<const WT*>(a.B) + (int64_t)(bare ? 0 : t.adapter) * a.N * a.rank;
  const int blocks = (a.N + kBlockCols - 1) / kBlockCols;
  const int c0 = blocks * share / a.shares + wave, c1 = blocks * (share + 1) / a.shares;
  if (c0 >= c1) return;
  auto load = [&](int c, Block<MT, YVEC>& y, BFrag<WT, RT>(&b)[4]) {
    const int n0 = c * kBlockCols;
    if (a.base)
      y.load(a.base, a.ldb, t.row0, t.rows, n0, a.N, r16, g);
    else
      y.zero();
    if (bare) return;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      b[u].load(B + (int64_t)min(n0 + block_col<YVEC>(u, r16), a.N - 1) * a.rank, ra, bvec, g);
  };
  Block<MT, YVEC> y, ny;
  BFrag<WT, RT> b[4], nb[4];
  load(c0, y, b);
  for (int c = c0; c < c1; c += NW) {
    if (c + NW < c1) load(c + NW, ny, nb);
    if (!bare) {
#pragma unroll
      for (int u = 0; u < 4; ++u) y.add(sf, b[u], u);
    }
    y.store(a.Y, a.ldy, t.row0, t.rows, c * kBlockCols, a.N, r16, g);
    y = ny;
#pragma unroll
    for (int u = 0; u < 4; ++u) b[u] = nb[u];
  }
}

// In two launches, for large outputs: k_lora_s computes S of every tile once and
// lays it out as the second product's operand; k_lora_expand adds S B^T to base.
// A streaming workgroup here has 256 columns of 32 rows only: workgroups that
// live short, started in address order, keep the chip's reads and writes in a
// narrow window of memory. A copy of a [16384, 8192] fp32 matrix with this
// kernel's accesses took 181 us with 256 columns a workgroup, 222 us with 2048
// and 254 us with whole rows (1024 columns: 199, a flat copy: 185).
//
// S lies in the workspace as the second product reads it: for every 16 rows of a
// tile SFrag's vectors, lane after lane.
template <typename WT, int RT>
constexpr int s_vectors() {
  return sizeof(WT) == 4 ? RT : SFrag<bf16, RT, 1>::KS;
}
constexpr int kExpandRows = 32, kExpandCols = 256;

template <typename XT, typename WT, int RT, int MT, int H, int NW>
__global__ __launch_bounds__(64 * NW) void k_lora_s(ForwardArgs a, bool xvec, v4f* s_rows,
                                                    int4* table) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int T = MT * 16, R = RT * 16, PARTS = kExpandRows / T;
  __shared__ __align__(16) SBuf<RT, MT, H, NW> buf;
  Tile t;
  const int tile = blockIdx.x / PARTS, part = blockIdx.x % PARTS;
  const bool found = find_tile(a.q, kExpandRows, tile, t);
  if (part == 0 && threadIdx.x == 0)
    table[tile] = found ? int4{t.row0, t.rows, t.adapter, 0} : int4{0, 0, -1, 0};
  if (!found || t.rows <= part * T || (t.adapter < 0 && !a.S)) return;
  t.row0 += part * T;
  t.rows = min(T, t.rows - part * T);
  const bool bare = t.adapter < 0;
  const int ra = bare ? 0 : rank_of(a.ranks, t.adapter, a.rank);
  const float sc = bare ? 0.0f : a.scales ? a.scales[t.adapter] : 1.0f;
  tile_s<XT, WT, RT, MT, H, NW>(a, t, ra, sc, xvec, a.S != nullptr, buf);
  if (bare) return;
  constexpr int V = s_vectors<WT, RT>();
  for (int m = wave; m < MT; m += NW) {
    SFrag<WT, RT, 1> f;
    f.load(&buf.v[0][m * 16][0], R + 4, lane & 15, lane >> 4);
    v4f* o = s_rows + ((int64_t)(tile * (kExpandRows / 16) + part * MT + m) * V) * kWave + lane;
#pragma unroll
    for (int k = 0; k < V; ++k) o[k * kWave] = __builtin_bit_cast(v4f, f.s[0][k]);
  }
}

template <typename WT, int RT, bool YVEC>
__global__ __launch_bounds__(256) void k_lora_expand(ForwardArgs a, bool bvec, const v4f* s_rows,
                                                     const int4* table) {
  constexpr int MT = kExpandRows / 16, V = s_vectors<WT, RT>();
  const int xcd = blockIdx.x & 7, loc = blockIdx.x >> 3;
  const int tile = loc / a.shares * 8 + xcd, share = loc % a.shares;
  const int4 t = table[tile];
  const int row0 = __builtin_amdgcn_readfirstlane(t.x), rows = __builtin_amdgcn_readfirstlane(t.y);
  const int ad = __builtin_amdgcn_readfirstlane(t.z);
  const bool bare = ad < 0;
  if (rows == 0 || (bare && a.base == a.Y)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, g = lane >> 4;
  const int n0 = share * kExpandCols + wave * kBlockCols;
  if (n0 >= a.N) return;
  Block<MT, YVEC> y;  // base first: it waits for nothing else
  if (a.base)
    y.load(a.base, a.ldb, row0, rows, n0, a.N, r16, g);
  else
    y.zero();
  if (!bare) {
    const int ra = rank_of(a.ranks, ad, a.rank);
    const WT* B = reinterpret_cast<const WT*>(a.B) + (int64_t)ad * a.N * a.rank;
    BFrag<WT, RT> b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      b[u].load(B + (int64_t)min(n0 + block_col<YVEC>(u, r16), a.N - 1) * a.rank, ra, bvec, g);
    SFrag<WT, RT, MT> sf;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int k = 0; k < V; ++k)
        sf.s[m][k] = __builtin_bit_cast(typename SFrag<WT, RT, MT>::vec,
                                        s_rows[((int64_t)(tile * MT + m) * V + k) * kWave + lane]);
#pragma unroll
    for (int u = 0; u < 4; ++u) y.add(sf, b[u], u);
  }
  y.store(a.Y, a.ldy, row0, rows, n0, a.N, r16, g);
}

// ------------------------------------------------------------------ dS = dY B ----
// One workgroup: a tile of MT * 16 rows and one split of the columns of dY. The
// waves take every NW-th 32 columns, the next step's loads ahead of this one's
// products, and join their sums in LDS. Lane l of a step has columns
// 8 (l / 16) .. + 7 of row l % 16 of dY, and rank l % 16 of the same rows of B.
// With bf16 B, dY goes in three bf16 terms: 16384 x 1152 at rank 64 with dB beside it
// took 88 us with fp32 instructions, 71 so (dB still in fp32 ones then).
//
// A single element of B as it is held until its use: bf16 in a register of its own
// (loads into register halves would wait for one another).
template <typename WT>
struct Held;
template <>
struct Held<float> {
  float v;
  __device__ __forceinline__ void load(const float* p) { v = *p; }
  __device__ __forceinline__ float get() const { return v; }
};
template <>
struct Held<bf16> {
  uint32_t v;
  __device__ __forceinline__ void load(const bf16* p) { v = *reinterpret_cast<const uint16_t*>(p); }
  __device__ __forceinline__ float get() const { return __uint_as_float(v << 16); }
};

template <int RT, int MT, int NW>
struct DsLds {
  float red[NW][MT * 16][RT * 16 + 4];
};

template <typename WT, int RT, int MT, int NW>
__device__ void ds_body(const DsArgs& a, int tile, int split, DsLds<RT, MT, NW>& lds) {
  constexpr int T = MT * 16;
  auto& red = lds.red;
  const bool vec = a.vec;
  Tile t;
  if (!find_tile(a.q, T, tile, t) || t.adapter < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, g = lane >> 4;
  const int c0 = split * a.split_len, c1 = min(a.N, c0 + a.split_len);
  const WT* B = reinterpret_cast<const WT*>(a.B) + (int64_t)t.adapter * a.N * a.rank;
  const float* prow[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    prow[m] = a.dY + (int64_t)(t.row0 + min(m * 16 + r16, t.rows - 1)) * a.ldy;
  int wj[RT];  // stored rank of this lane (clamped: its sums are dropped at the end)
#pragma unroll
  for (int r = 0; r < RT; ++r) wj[r] = min(r * 16 + r16, a.rank - 1);
  v4f acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[m][r] = v4f{0, 0, 0, 0};
  Frag8<float> x[MT], nx[MT];
  Held<WT> w[RT][8], nw[RT][8];
  auto load = [&](int c, Frag8<float>(&fx)[MT], Held<WT>(&fw)[RT][8]) {
    const int k = c + 8 * g, valid = c1 - k;
    if (vec && c + kDsStep <= c1) {
#pragma unroll
      for (int m = 0; m < MT; ++m) fx[m].load(prow[m] + k);
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int r = 0; r < RT; ++r) fw[r][e].load(B + (int64_t)(k + e) * a.rank + wj[r]);
      return;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) fx[m].load(prow[m] + k, valid);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // past the end dY is zero; the row of B read there is the last one, whose
      // elements may not be finite, so it is zero too
      const WT* row = B + (int64_t)min(k + e, a.N - 1) * a.rank;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        fw[r][e].load(row + wj[r]);
        if (e >= valid) fw[r][e].v = 0;
      }
    }
  };
  int c = c0 + wave * kDsStep;
  if (c < c1) load(c, x, w);
  for (; c < c1; c += NW * kDsStep) {
    if (c + NW * kDsStep < c1) load(c + NW * kDsStep, nx, nw);
    if constexpr (sizeof(WT) == 2) {  // dY in three bf16 terms, B as it is
      v8h wf[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = w[r][2 * e].v | (w[r][2 * e + 1].v << 16);
        __builtin_memcpy(&wf[r], u, 16);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        v8h h, mi, l;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          bf16 p, q, o;
          split3(x[m].get(e), p, q, o);
          h[e] = p;
          mi[e] = q;
          l[e] = o;
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          acc[m][r] = mfma_bf16(wf[r], h, acc[m][r]);
          acc[m][r] = mfma_bf16(wf[r], mi, acc[m][r]);
          acc[m][r] = mfma_bf16(wf[r], l, acc[m][r]);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int r = 0; r < RT; ++r) acc[m][r] = mfma_f32(w[r][e].get(), x[m].get(e), acc[m][r]);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) x[m] = nx[m];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 8; ++e) w[r][e] = nw[r][e];
  }
  // acc[m][r][i]: row 16 m + lane % 16, rank 16 r + 4 g + i
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < RT; ++r)
      *reinterpret_cast<v4f*>(&red[wave][m * 16 + r16][r * 16 + 4 * g]) = acc[m][r];
  __syncthreads();
  const int ra = rank_of(a.ranks, t.adapter, a.rank);
  const float sc = a.scales ? a.scales[t.adapter] : 1.0f;
  float* out = a.part + ((int64_t)split * a.q.rows + t.row0) * a.rank;
  for (int u = threadIdx.x; u < t.rows * a.rank; u += 64 * NW) {
    const int row = u / a.rank, j = u % a.rank;
    float v = red[0][row][j];
#pragma unroll
    for (int k = 1; k < NW; ++k) v += red[k][row][j];
    out[u] = j < ra ? v * sc : 0.0f;
  }
}

// ------------------------------------------------------------------- outer ----
// dA_a = dS^T X with dX = dS A_a on the way (one reading of X), and dB_a = dY^T S.
// One workgroup: 256 columns (32 a wave) of one range of rows, 32 rows at a time.
// Q (dS or S, rank values a row) goes through LDS, double-buffered; piece by piece
// (the rows of one request in the range) Q^T P is summed in registers and written to
// a slot of its own, and A's columns stay in registers for the whole range. Long
// ranges keep the slots few: they are written and read once more, D * rank * 4 bytes
// each.
//
// bf16 P (or bf16 results) take bf16 matrix instructions, whose operands run along
// the rows: LDS is read transposed (ds_read_b64_tr_b16: lane c of 16 gets four rows
// of column c). fp32 P comes element by element from memory, lanes side by side at
// addresses side by side: split in registers for bf16 results, as it is for fp32.
//
// Measured at 16384 rows, K 4608, rank 64, bf16: 109-118 us for 302 MB of X and dX and
// 40 MB of slots, 3 TB/s (with 16 bits of dS instead of 24 it was 97); bound by the rows'
// latency between barriers, with one workgroup a compute unit to wait for them. Four
// waves of 64 columns instead of eight of 32: 268 instead of 231 us for the whole
// gradient then; 256 threads and 128 columns: 260 instead of 200.
constexpr int kOuterRows = 32, kOuterThreads = 512;
constexpr int kOuterU = 2;  // 16-column tiles of a wave
constexpr int kOuterCols = kOuterThreads / 64 * 16 * kOuterU;

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s* lds_v4s;

// Rows 4 g .. + 3 and 16 + 4 g .. + 3 of column lane % 16 of a [32][ld] tile of bf16.
__device__ __forceinline__ v8h read_transposed(const bf16* tile, int ld, int r16, int g) {
  const bf16* p = tile + (4 * g + r16 / 4) * ld + 4 * (r16 % 4);
  const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p));
  const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p + 16 * ld));
  return __builtin_bit_cast(v8h, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

template <typename PT, typename WT, int RT, bool DX>
struct OuterLds {
  static constexpr int R = RT * 16;
  static constexpr int XLD = kOuterCols + 8, QLD = R + 8, FLD = R + 16;
  static constexpr bool PB = sizeof(PT) == 2;  // bf16 products for Q^T P, P through LDS
  static constexpr bool PS = !PB && sizeof(WT) == 2;  // the same, fp32 P split in registers
  static constexpr bool XB = DX && sizeof(WT) == 2;  // bf16 products for dX
  static constexpr bool kSplit = PB || PS || XB;  // bf16 products read Q's three terms
  static constexpr bool kFloat = (!PB && !PS) || (DX && !XB);  // fp32 products read Q itself
  static constexpr int kPlanes = !kSplit ? 0 : RT == 1 && XB ? 4 : 3;
  struct Tile {
    float q[kFloat ? kOuterRows : 1][FLD];
    bf16 x[PB ? kOuterRows : 1][XLD];
    bf16 h[kPlanes ? kPlanes : 1][kPlanes ? kOuterRows : 1][QLD];  // (a fourth one of zeros)
  };
  Tile tile[2];  // one is used while the next is written
};

template <typename PT, typename WT, int RT, bool DX, bool TR>
__device__ void outer_body(const OuterArgs& a, int chunk, int sp, OuterLds<PT, WT, RT, DX>& lds) {
  typedef OuterLds<PT, WT, RT, DX> L;
  constexpr int R = RT * 16, U = kOuterU;
  constexpr bool PB = L::PB, PS = L::PS, XB = L::XB;
  constexpr int t_xld = L::XLD, t_qld = L::QLD, t_fld = L::FLD;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, g = lane >> 4;
  const int dw = chunk * kOuterCols, d0 = dw + wave * 16 * U;  // the workgroup's, the wave's columns
  const int lo = min(sp * a.row_len, a.q.rows), hi = min(lo + a.row_len, a.q.rows);
  const PT* P = reinterpret_cast<const PT*>(a.P);
  PT* dX = reinterpret_cast<PT*>(a.dX);
  const int64_t qstride = (int64_t)a.q.rows * a.rank;
  // Requests first .. last touch this range (ends included, so that the slots
  // s + i of neighbouring ranges join without gaps).
  int first = 0, last = a.q.n - 1;
  {
    int cl = 0, ch = 0;  // requests that end at or before lo / hi
    for (int base = 0; base < a.q.n; base += kWave) {
      const int i = base + lane;
      const int e = i < a.q.n ? clampi(a.q.off[i + 1], 0, a.q.rows) : 0x7fffffff;
      cl += __popcll(__ballot(e <= lo));
      ch += __popcll(__ballot(e <= hi));
    }
    if (sp > 0) first = min(cl, a.q.n - 1);
    if (sp + 1 < a.splits) last = min(ch, a.q.n - 1);
  }
  v4f acc[RT][U];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int u = 0; u < U; ++u) acc[r][u] = v4f{0, 0, 0, 0};
  BFrag<WT, RT> af[U];  // A's columns d0 + col(u), like rows of B
  int af_of = -1;
  bool pending = false;
  const auto col = [&](int u) { return U * r16 + u; };
  // Row of element k of a lane: split P's must be those of read_transposed.
  const auto p_row = [&](int k) { return PS ? (k < 4 ? 4 * g + k : 12 + 4 * g + k) : 4 * k + g; };
  for (int i = first; i <= last; ++i) {
    const int b = clampi(a.q.off[i], 0, a.q.rows), e = clampi(a.q.off[i + 1], b, a.q.rows);
    const int r0 = max(b, lo), r1 = min(e, hi);
    const int id = a.q.ids[i];
    const int ad = id >= 0 && id < a.q.n_adapters ? id : -1;
    if (r0 < r1 && ad >= 0) {
      const int ra = rank_of(a.ranks, ad, a.rank);
      // this thread's part of a tile: Q values and, for bf16 P, 16-byte pieces of P
      // Addresses are clamped into the piece and what lies past it is zeroed when
      // the tile is used: the loads wait for nothing and nothing waits for them.
      constexpr int QN = kOuterRows * R / kOuterThreads, QW = QN < 4 ? QN : 4;
      constexpr int XP = kOuterCols / 8, XN = PB ? kOuterRows * XP / kOuterThreads : 1;
      typedef float vq __attribute__((ext_vector_type(QW)));
      const int qm = threadIdx.x * QN / R, qj = threadIdx.x * QN % R;
      vq qr[QN / QW];
      v8h xr[XN];
      PT pr[PB ? 1 : 8][PB ? 1 : U];
      auto fetch_q = [&](int m0, int split, vq(&v)[QN / QW]) {
        const float* qp = a.part + split * qstride + (int64_t)min(m0 + qm, r1 - 1) * a.rank;
#pragma unroll
        for (int k = 0; k < QN / QW; ++k) {
          if (a.q_vec) {
            const int j = qj + k * QW;
            v[k] = *reinterpret_cast<const vq*>(qp + (j < a.rank ? j : 0));
          } else {
#pragma unroll
            for (int c = 0; c < QW; ++c) v[k][c] = qp[min(qj + k * QW + c, a.rank - 1)];
          }
        }
      };
      auto fetch = [&](int m0) {
        fetch_q(m0, 0, qr);
        if constexpr (PB) {
#pragma unroll
          for (int k = 0; k < XN; ++k) {
            const int v = k * kOuterThreads + threadIdx.x, d = dw + v % XP * 8;
            // D % 8 == 0 for bf16 P
            const PT* p = P + (int64_t)min(m0 + v / XP, r1 - 1) * a.ldp + min(d, a.D - 8);
            if (a.p_vec) {
              xr[k] = *reinterpret_cast<const v8h*>(p);
            } else {
#pragma unroll
              for (int c = 0; c < 8; ++c) xr[k][c] = p[c];
            }
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const PT* p = P + (int64_t)min(m0 + p_row(kk), r1 - 1) * a.ldp;
#pragma unroll
            for (int u = 0; u < U; ++u) pr[kk][u] = p[min(d0 + 16 * u + r16, a.D - 1)];
          }
        }
      };
      // Puts the fetched tile into LDS (and, for fp32 P, into pc).
      float pc[PB ? 1 : 8][PB ? 1 : U];
      auto put = [&](int m0, typename L::Tile& t) {
        float qz[QN];
#pragma unroll
        for (int k = 0; k < QN; ++k) qz[k] = qr[k / QW][k % QW];
        for (int sq = 1; sq < a.q_splits; ++sq) {
          vq more[QN / QW];
          fetch_q(m0, sq, more);
#pragma unroll
          for (int k = 0; k < QN; ++k) qz[k] += more[k / QW][k % QW];
        }
#pragma unroll
        for (int k = 0; k < QN; ++k)
          if (m0 + qm >= r1 || qj + k >= ra) qz[k] = 0.0f;
        if constexpr (L::kFloat) {
#pragma unroll
          for (int k = 0; k < QN; ++k) t.q[qm][qj + k] = qz[k];
        }
        if constexpr (L::kSplit) {
          typedef bf16 vt __attribute__((ext_vector_type(QN < 8 ? QN : 8)));
          constexpr int W = QN < 8 ? QN : 8;
#pragma unroll
          for (int c = 0; c < QN / W; ++c) {
            vt h, mi, l;
#pragma unroll
            for (int k = 0; k < W; ++k) {
              bf16 x, y, z;
              split3(qz[c * W + k], x, y, z);
              h[k] = x;
              mi[k] = y;
              l[k] = z;
            }
            *reinterpret_cast<vt*>(&t.h[0][qm][qj + c * W]) = h;
            *reinterpret_cast<vt*>(&t.h[1][qm][qj + c * W]) = mi;
            *reinterpret_cast<vt*>(&t.h[2][qm][qj + c * W]) = l;
            if constexpr (RT == 1 && XB) *reinterpret_cast<vt*>(&t.h[3][qm][qj]) = vt(0.0f);
          }
        }
        if constexpr (PB) {
#pragma unroll
          for (int k = 0; k < XN; ++k) {
            const int v = k * kOuterThreads + threadIdx.x, m = v / XP, c = v % XP * 8;
            const bool in = m0 + m < r1 && dw + c < a.D;
            *reinterpret_cast<v8h*>(&t.x[m][c]) = in ? xr[k] : v8h(0.0f);
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
#pragma unroll
            for (int u = 0; u < U; ++u)
              pc[kk][u] = m0 + p_row(kk) < r1 && d0 + 16 * u + r16 < a.D ? (float)pr[kk][u] : 0.0f;
        }
      };
      __syncthreads();  // the last piece's tiles have been read
      fetch(r0);
      if (DX && af_of != ad) {
        af_of = ad;
        const WT* A = reinterpret_cast<const WT*>(a.A) + (int64_t)ad * a.rank * a.D;
#pragma unroll
        for (int u = 0; u < U; ++u)
          af[u].load_column(A + min(d0 + col(u), a.D - 1), a.D, ra, g);
      }
      put(r0, lds.tile[0]);
      fetch(r0 + kOuterRows);
      int cur = 0;
      for (int m0 = r0; m0 < r1; m0 += kOuterRows, cur ^= 1) {
        __syncthreads();  // tile `cur` is written, the other one has been read
        const auto& t = lds.tile[cur];
        if constexpr (PB) {
          v8h xt[U];
#pragma unroll
          for (int u = 0; u < U; ++u)
            xt[u] = read_transposed(&t.x[0][wave * 16 * U + 16 * u], t_xld, r16, g);
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              const v8h qt = read_transposed(&t.h[k][0][16 * r], t_qld, r16, g);
#pragma unroll
              for (int u = 0; u < U; ++u) acc[r][u] = mfma_bf16(qt, xt[u], acc[r][u]);
            }
        } else if constexpr (PS) {
          v8h ph[U], pm[U], pl[U];
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              bf16 h, m, l;
              split3(pc[k][u], h, m, l);
              ph[u][k] = h;
              pm[u][k] = m;
              pl[u][k] = l;
            }
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const v8h qh = read_transposed(&t.h[0][0][16 * r], t_qld, r16, g);
            const v8h qm = read_transposed(&t.h[1][0][16 * r], t_qld, r16, g);
            const v8h ql = read_transposed(&t.h[2][0][16 * r], t_qld, r16, g);
#pragma unroll
            for (int u = 0; u < U; ++u) {
              auto add = [&](const v8h& q, const v8h& p) {
                acc[r][u] = TR ? mfma_bf16(q, p, acc[r][u]) : mfma_bf16(p, q, acc[r][u]);
              };
              // all but the products below 2^-24 of the first
              add(qh, ph[u]);
              add(qm, ph[u]);
              add(qh, pm[u]);
              add(qm, pm[u]);
              add(ql, ph[u]);
              add(qh, pl[u]);
            }
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              const float qv = t.q[kk * 4 + g][16 * r + r16];
#pragma unroll
              for (int u = 0; u < U; ++u)
                acc[r][u] = TR ? mfma_f32(qv, pc[kk][u], acc[r][u]) : mfma_f32(pc[kk][u], qv, acc[r][u]);
            }
        }
        if constexpr (DX) {
#pragma unroll
          for (int m = 0; m < kOuterRows / 16; ++m) {
            v4f y[U];
            if constexpr (XB) {
              constexpr int KS = SFrag<bf16, RT, 1>::KS;
#pragma unroll
              for (int u = 0; u < U; ++u) y[u] = v4f{0, 0, 0, 0};
#pragma unroll
              for (int k = 0; k < KS; ++k) {
                const int plane = RT == 1 ? 2 * k + g / 2 : k % 3;
                const int j = RT == 1 ? 8 * (g & 1) : 32 * (k / 3) + 8 * g;
                const v8h sv = *reinterpret_cast<const v8h*>(&t.h[plane][m * 16 + r16][j]);
#pragma unroll
                for (int u = 0; u < U; ++u)
                  y[u] = mfma_bf16(sv, af[u].b[RT == 1 ? 0 : k / 3], y[u]);
              }
            } else {
              SFrag<WT, RT, 1> sf;
              sf.load(&t.q[m * 16][0], t_fld, r16, g);
#pragma unroll
              for (int u = 0; u < U; ++u) y[u] = af[u].times(sf, 0);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = m0 + m * 16 + 4 * g + k, d = d0 + col(0);
              if (row >= r1 || d >= a.D) continue;  // D % 16 == 0 for dX
              PT* o = dX + (int64_t)row * a.lddx + d;
              typedef PT vu __attribute__((ext_vector_type(U)));
              vu v;
#pragma unroll
              for (int u = 0; u < U; ++u) v[u] = (PT)y[u][k];
              if (a.dx_vec) {
                *reinterpret_cast<vu*>(o) = v;
              } else {
#pragma unroll
                for (int u = 0; u < U; ++u) o[u] = v[u];
              }
            }
          }
        }
        if (m0 + kOuterRows < r1) {
          put(m0 + kOuterRows, lds.tile[cur ^ 1]);
          fetch(m0 + 2 * kOuterRows);  // past the end: the last row again, unused
        }
      }
      pending = true;
    } else if (DX && r0 < r1) {  // no adapter: zero rows
      for (int v = threadIdx.x; v < (r1 - r0) * kOuterCols; v += kOuterThreads) {
        const int d = dw + v % kOuterCols;
        if (d < a.D) dX[(int64_t)(r0 + v / kOuterCols) * a.lddx + d] = (PT)0.0f;
      }
    }
    // Write the sum unless the next request goes on with the same adapter.
    const bool flush = pending && (i == last || a.q.ids[i + 1] != id);
    if (chunk == 0 && threadIdx.x == 0) a.slot_id[sp + i] = flush ? ad : -1;
    if (flush) {
      float* out = a.out + (int64_t)(sp + i) * a.D * a.rank;
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int j = TR ? r * 16 + 4 * g + k : r * 16 + r16;
            const int d = d0 + 16 * u + (TR ? r16 : 4 * g + k);
            if (j < a.rank && d < a.D)
              out[TR ? (int64_t)j * a.D + d : (int64_t)d * a.rank + j] = acc[r][u][k];
          }
          acc[r][u] = v4f{0, 0, 0, 0};
        }
      pending = false;
    }
  }
}

// What needs dY alone, in one launch: dB in workgroups [0, y_groups), which run
// longest, dS in the rest. Both wait for memory more than they compute, and what one
// reads of dY the other finds in the caches. 60-64 us at 16384 x 1152, rank 64 (75 MB
// of dY; dS first instead of dB: 99 against 88 us before both went to bf16).
template <typename WT, int RT, int MT>
__global__ __launch_bounds__(kOuterThreads) void k_lora_grad_y(DsArgs d, OuterArgs y, int y_groups) {
  __shared__ __align__(16) union Lds {
    DsLds<RT, MT, kOuterThreads / 64> d;
    OuterLds<float, WT, RT, false> y;
    __device__ Lds() {}
  } lds;
  const int id = blockIdx.x;
  if (id < y_groups)
    outer_body<float, WT, RT, false, false>(y, id % y.chunks, id / y.chunks, lds.y);
  else
    ds_body<WT, RT, MT, kOuterThreads / 64>(d, (id - y_groups) / d.splits, (id - y_groups) % d.splits,
                                            lds.d);
}

// What needs X and dS: dA and dX.
template <typename XT, typename WT, int RT, bool DX>
__global__ __launch_bounds__(kOuterThreads) void k_lora_grad_x(OuterArgs x) {
  __shared__ __align__(16) OuterLds<XT, WT, RT, DX> lds;
  outer_body<XT, WT, RT, DX, true>(x, blockIdx.x % x.chunks, blockIdx.x / x.chunks, lds);
}

// ---------------------------------------------------------------- slot sum ----
// dW[a][e] = scale_a * the sum of the slots of adapter a, in the slots' order. Bound
// by memory (55 MB of slots in 13 us at 16384 rows, rank 64): eight loads at a time,
// 4.5 us for 32 slots of 92160 values where one after another took 9.
template <typename WT>
__global__ __launch_bounds__(256) void k_lora_slot_sum(SlotSumArgs p, SlotSumArgs s, int p_groups) {
  const bool second = (int)blockIdx.x >= p_groups;
  const SlotSumArgs& a = second ? s : p;
  const int64_t len = (int64_t)a.D * a.rank;
  const int64_t e = (int64_t)(second ? blockIdx.x - p_groups : blockIdx.x) * 256 + threadIdx.x;
  const int ad = blockIdx.y, lane = threadIdx.x & 63;
  float v = 0.0f;
  for (int base = 0; base < a.slots; base += kWave) {
    const int i = base + lane;
    uint64_t hit = __ballot(i < a.slots && a.slot_id[i] == ad);
    while (hit) {  // eight slots' loads at a time
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool any = hit != 0;
        const int at = base + (any ? __ffsll((unsigned long long)hit) - 1 : 0);
        hit &= hit - 1;
        x[k] = any && e < len ? a.part[at * len + e] : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) v += x[k];
    }
  }
  if (e >= len) return;
  const int j = a.transposed ? (int)(e / a.D) : (int)(e % a.rank);
  const float sc = a.scales ? a.scales[ad] : 1.0f;
  const float r = j < rank_of(a.ranks, ad, a.rank) ? v * sc : 0.0f;
  reinterpret_cast<WT*>(a.out)[ad * len + e] = (WT)r;
}

int max_tiles(const Requests& q, int T) {
  const int64_t t = (int64_t)q.rows / T + q.n;
  return (int)(t < q.rows ? t : q.rows);
}

// Calls with fewer outputs than this take one launch. Measured (one launch / two):
// 1024 x 4608, K 1152, rank 16, fp32: 15.3 / 17.9 us; 1024 x 4608, K 2048, rank 64,
// bf16: 21.9 / 24.8; guided 2048 x 4608, K 1152, rank 16, fp32: 38.4 / 27.5;
// 16384 x 8192, K 2048, rank 64, bf16: 298 / 239.
constexpr int64_t kTwoLaunches = 1 << 23;
bool two_launches(int rows, int N) { return (int64_t)rows * N >= kTwoLaunches; }

// Padded tiles of the two-launch form.
int expand_tiles(int rows, int n_req) {
  Requests q{};
  q.rows = rows;
  q.n = n_req;
  return (max_tiles(q, kExpandRows) + 7) / 8 * 8;
}
// Bytes of S of one tile.
int64_t s_bytes(int rank, bool w_bf16) {
  const int rt = rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8;
  const int vectors = !w_bf16 ? rt : rt == 1 ? 2 : 3 * rt / 2;
  return (int64_t)(kExpandRows / 16) * vectors * kWave * 16;
}

template <typename XT, typename WT, int RT, int H>
hipError_t forward_run(ForwardArgs a, hipStream_t s) {
  const bool xvec = reinterpret_cast<uintptr_t>(a.X) % 16 == 0 && (a.ldx * sizeof(XT)) % 16 == 0;
  const bool yvec = reinterpret_cast<uintptr_t>(a.Y) % 16 == 0 && a.ldy % 4 == 0 &&
                    (!a.base || (reinterpret_cast<uintptr_t>(a.base) % 16 == 0 && a.ldb % 4 == 0));
  const bool bvec = reinterpret_cast<uintptr_t>(a.B) % 16 == 0 && a.rank % (16 / sizeof(WT)) == 0;
  if (two_launches(a.q.rows, a.N)) {
    // S by 32 rows a workgroup reads A half as often as by 16; used where registers
    // and LDS hold it and the tiles fill the chip. Measured by 32 / 16 rows on 16384
    // rows: K 2048, N 8192, rank 64, bf16 238 / 254 us; K 1152, N 4608, rank 32 135.5 /
    // 137.7 us, rank 16, fp32 129.7 / 129.7 us.
    constexpr bool kTall = RT * H <= 4;
    const int tiles = expand_tiles(a.q.rows, a.q.n);
    int4* table = reinterpret_cast<int4*>(a.ws);
    v4f* s_rows = reinterpret_cast<v4f*>(table + tiles);
    if (kTall && tiles >= 512)
      hipLaunchKernelGGL((k_lora_s<XT, WT, RT, kTall ? 2 : 1, H, 8>), dim3(tiles), dim3(512), 0, s, a,
                         xvec, s_rows, table);
    else
      hipLaunchKernelGGL((k_lora_s<XT, WT, RT, 1, H, 8>), dim3(2 * tiles), dim3(512), 0, s, a, xvec,
                         s_rows, table);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.shares = (a.N + kExpandCols - 1) / kExpandCols;
    const dim3 grid(tiles * a.shares);
    if (yvec)
      hipLaunchKernelGGL((k_lora_expand<WT, RT, true>), grid, dim3(256), 0, s, a, bvec, s_rows,
                         table);
    else
      hipLaunchKernelGGL((k_lora_expand<WT, RT, false>), grid, dim3(256), 0, s, a, bvec, s_rows,
                         table);
    return hipGetLastError();
  }
  constexpr int NW = 8;
  const int tiles = (max_tiles(a.q, 16) + 7) / 8 * 8;
  // About one workgroup a compute unit: more of them would compute S again (512
  // instead of 256: 1003 ragged rows 14.7 instead of 12.0 us).
  const int want = (256 + tiles - 1) / tiles, cap = (a.N + 127) / 128;
  a.shares = want < cap ? want : cap;
  const dim3 grid(tiles * a.shares), block(64 * NW);
  if (yvec)
    hipLaunchKernelGGL((k_lora_forward<XT, WT, RT, 1, H, NW, true>), grid, block, 0, s, a, xvec,
                       bvec);
  else
    hipLaunchKernelGGL((k_lora_forward<XT, WT, RT, 1, H, NW, false>), grid, block, 0, s, a, xvec,
                       bvec);
  return hipGetLastError();
}

template <typename XT, typename WT>
hipError_t forward_rt(const ForwardArgs& a, hipStream_t s) {
#define QL_RUN(RT) \
  (a.halves == 2 ? forward_run<XT, WT, RT, 2>(a, s) : forward_run<XT, WT, RT, 1>(a, s))
  if (a.rank <= 16) return QL_RUN(1);
  if (a.rank <= 32) return QL_RUN(2);
  if (a.rank <= 64) return QL_RUN(4);
  return QL_RUN(8);
#undef QL_RUN
}

bool q_vec(const OuterArgs& o) {
  return reinterpret_cast<uintptr_t>(o.part) % 16 == 0 && o.rank % 4 == 0;
}

template <typename WT, int RT>
hipError_t grad_y_run(DsArgs d, OuterArgs y, hipStream_t s) {
  constexpr int MT = RT == 8 ? 1 : 2;  // rows of a tall tile: the waves' sums fit LDS
  d.vec = reinterpret_cast<uintptr_t>(d.dY) % 16 == 0 && d.ldy % 4 == 0;
  y.chunks = (y.D + kOuterCols - 1) / kOuterCols;
  y.q_vec = q_vec(y);
  const int yg = y.out ? y.chunks * y.splits : 0;
  const bool tall = d.tall && MT == 2;
  const int dg = d.part ? max_tiles(d.q, tall ? 32 : 16) * d.splits : 0;
  if (tall)
    hipLaunchKernelGGL((k_lora_grad_y<WT, RT, MT>), dim3(dg + yg), dim3(kOuterThreads), 0, s, d, y, yg);
  else
    hipLaunchKernelGGL((k_lora_grad_y<WT, RT, 1>), dim3(dg + yg), dim3(kOuterThreads), 0, s, d, y, yg);
  return hipGetLastError();
}

template <typename XT, typename WT, int RT>
hipError_t grad_x_run(OuterArgs x, hipStream_t s) {
  x.chunks = (x.D + kOuterCols - 1) / kOuterCols;
  x.p_vec = reinterpret_cast<uintptr_t>(x.P) % 16 == 0 && (x.ldp * sizeof(XT)) % 16 == 0;
  x.q_vec = q_vec(x);
  x.dx_vec = reinterpret_cast<uintptr_t>(x.dX) % (kOuterU * sizeof(XT)) == 0 && x.lddx % kOuterU == 0;
  const dim3 grid(x.chunks * x.splits), block(kOuterThreads);
  if (x.dX)
    hipLaunchKernelGGL((k_lora_grad_x<XT, WT, RT, true>), grid, block, 0, s, x);
  else
    hipLaunchKernelGGL((k_lora_grad_x<XT, WT, RT, false>), grid, block, 0, s, x);
  return hipGetLastError();
}

template <typename XT, typename WT>
hipError_t grad_x_rt(const OuterArgs& x, hipStream_t s) {
  if (x.rank <= 16) return grad_x_run<XT, WT, 1>(x, s);
  if (x.rank <= 32) return grad_x_run<XT, WT, 2>(x, s);
  if (x.rank <= 64) return grad_x_run<XT, WT, 4>(x, s);
  return grad_x_run<XT, WT, 8>(x, s);
}

template <typename WT>
hipError_t grad_y_rt(const DsArgs& d, const OuterArgs& y, hipStream_t s) {
  if (y.rank <= 16) return grad_y_run<WT, 1>(d, y, s);
  if (y.rank <= 32) return grad_y_run<WT, 2>(d, y, s);
  if (y.rank <= 64) return grad_y_run<WT, 4>(d, y, s);
  return grad_y_run<WT, 8>(d, y, s);
}

}  // namespace

// Tall tiles (32 rows) read B half as often; used where they still fill the
// chip. Otherwise 16 rows, and the columns of dY split over workgroups.
bool lora_ds_tall(int rows, int n_req) { return (int64_t)rows / 32 + n_req >= 256; }

int lora_ds_splits(int rows, int n_req, int N) {
  if (lora_ds_tall(rows, n_req)) return 1;
  const int64_t tiles = (int64_t)rows / 16 + n_req;
  int64_t s = 256 / tiles;
  const int64_t cap = N / 512;
  s = s < cap ? s : cap;
  return (int)(s < 1 ? 1 : s > 8 ? 8 : s);
}

// Row ranges: at most `groups` workgroups, none with fewer than 64 rows. Workgroups
// here take long and alike, so they are counted to fill the chip evenly, in whole
// rounds: two a compute unit are resident up to rank 16, one at rank 64 (222 registers
// on the X side, 186 on the dY side). On the X side 504 of them instead of 774 took 171
// instead of 195 us for the whole gradient at 16384 rows, rank 64 (1008: 192). On the
// dY side dB gets what dS leaves of the next multiple of 256 (96 at least): 16384 rows
// 171 us against 178 with 256 of them, 2048 rows, N 4608, rank 16, fp32 35.9 against 39.0.
constexpr int kXGroups = 512;
static int outer_splits(int rows, int D, int groups) {
  const int chunks = (D + kOuterCols - 1) / kOuterCols;
  int64_t s = groups / chunks;
  const int64_t cap = (rows + 63) / 64;
  s = s < cap ? s : cap;
  return (int)(s < 1 ? 1 : s);
}
int lora_x_splits(int rows, int K) { return outer_splits(rows, K, kXGroups); }
int lora_y_splits(int rows, int n_req, int N) {
  const int64_t ds = lora_ds_tall(rows, n_req)
                         ? (int64_t)rows / 32 + n_req
                         : ((int64_t)rows / 16 + n_req) * lora_ds_splits(rows, n_req, N);
  const int64_t all = (ds + 96 + 255) / 256 * 256;
  return outer_splits(rows, N, (int)(all - ds));
}

// A launch holds fewer than 2^32 threads along its grid. The gradient's dY side has
// a workgroup for every tile of rows (or at most 256) and, beside them, 352 at most or
// one for every chunk of N.
bool lora_fits(int rows, int n_req, int N, bool grad) {
  Requests q{};
  q.rows = rows;
  q.n = n_req;
  const int64_t chunks = ((int64_t)N + kOuterCols - 1) / kOuterCols + 256;
  int64_t threads = ((int64_t)max_tiles(q, 16) + (grad && chunks > 512 ? chunks : 512)) * 512;
  if (!grad && two_launches(rows, N)) {
    const int64_t shares = ((int64_t)N + kExpandCols - 1) / kExpandCols;
    threads = expand_tiles(rows, n_req) * (shares > 4 ? shares : 4) * 256;
  }
  return threads < (int64_t)1 << 32;
}

int64_t lora_forward_ws(int rows, int n_req, int N, int rank, bool w_bf16) {
  if (!two_launches(rows, N)) return 0;
  return expand_tiles(rows, n_req) * ((int64_t)sizeof(int4) + s_bytes(rank, w_bf16));
}

hipError_t launch_lora_forward(const ForwardArgs& a, hipStream_t s) {
  if (a.x_bf16) return a.w_bf16 ? forward_rt<bf16, bf16>(a, s) : forward_rt<bf16, float>(a, s);
  return a.w_bf16 ? forward_rt<float, bf16>(a, s) : forward_rt<float, float>(a, s);
}

hipError_t launch_lora_grad_y(const DsArgs& d, const OuterArgs& y, hipStream_t s) {
  return y.w_bf16 ? grad_y_rt<bf16>(d, y, s) : grad_y_rt<float>(d, y, s);
}

hipError_t launch_lora_grad_x(const OuterArgs& x, hipStream_t s) {
  if (x.p_bf16) return x.w_bf16 ? grad_x_rt<bf16, bf16>(x, s) : grad_x_rt<bf16, float>(x, s);
  return x.w_bf16 ? grad_x_rt<float, bf16>(x, s) : grad_x_rt<float, float>(x, s);
}

hipError_t launch_lora_slot_sum(const SlotSumArgs& p, const SlotSumArgs& q, hipStream_t s) {
  auto groups = [](const SlotSumArgs& a) {
    return a.out ? (unsigned)(((int64_t)a.D * a.rank + 255) / 256) : 0u;
  };
  const dim3 grid(groups(p) + groups(q), q.n_adapters);
  if (q.w_bf16)
    hipLaunchKernelGGL(k_lora_slot_sum<bf16>, grid, dim3(256), 0, s, p, q, (int)groups(p));
  else
    hipLaunchKernelGGL(k_lora_slot_sum<float>, grid, dim3(256), 0, s, p, q, (int)groups(p));
  return hipGetLastError();
}

}  // namespace ql
