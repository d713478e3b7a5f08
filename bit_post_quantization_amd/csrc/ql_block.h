// Internal interface between the C ABI of a conditioned block's operators
// (qlinear_block.cpp) and their kernels (k_rows4.hip, k_heads.hip, k_attn.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/qlinear.h"

namespace ql {

// Before launches of a kernel with more than 64 KB of LDS: its limit of dynamic LDS, once a
// device, to the most that any of its calls asks for. The limit is the kernel's, shared by all
// host threads: one that sets it to its own call's need could lower it between another's
// setting and launch.
template <auto Kernel, int Bytes>
hipError_t allow_lds() {
  static std::atomic<uint64_t> devices{0};
  int device = 0;
  hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) return e;
  const uint64_t bit = device < 64 ? (uint64_t)1 << device : 0;
  if (devices.load(std::memory_order_relaxed) & bit) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(Kernel),
                          hipFuncAttributeMaxDynamicSharedMemorySize, Bytes);
  if (e == hipSuccess) devices.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// -------------------------------------------------------------- 4-bit rows ----

// Weights as the kernel reads them: tiles of 16 output channels by units of 128 input
// channels, tile after tile. A unit is 64 pieces of 16 bytes, word s of piece 16 q + i
// holding the codes of channel 16 tile + i at inputs 32 s + 8 q .. + 7 (nibble j: input
// j of the eight). Behind the codes the scales, [tile][group][16], with groups up to the
// end of the last unit.
struct Rows4Layout {
  int tiles, units, groups, spots;  // spots: groups with those past K
  int64_t scales, bytes;            // offset of the scales, bytes in all
};
Rows4Layout rows4_layout(const ql_rows4& d);

typedef uint32_t Rows4Piece __attribute__((ext_vector_type(4)));
struct Rows4Args {
  const Rows4Piece* codes;
  const void* scales;
  const float* bias;
  const void* X;
  int64_t ldx;
  float* Y;
  int64_t ldy;
  char* digits;   // workspace: act(X) in fixed point
  float* worths;  // workspace: [M][units]
  float* part;    // workspace: [splits][M][N], splits > 1
  int M, N, K, units, tiles, group;
  int splits;     // workgroups that share a tile's inputs (set by the launch)
  bool x_bf16, s_bf16, silu;
  bool x_vec;     // rows of X are 16-byte aligned
};
struct Rows4Ws {
  int64_t worths, part, bytes;  // offsets, and bytes in all
};
Rows4Ws rows4_ws(const ql_rows4& d, int M);
hipError_t launch_rows4(const Rows4Args& a, hipStream_t s);
hipError_t launch_rows4_pack(const ql_rows4& d, const int8_t* codes, const void* scales,
                             void* packed, hipStream_t s);
hipError_t launch_rows4_quantize(const ql_rows4& d, const void* W, bool w_bf16, void* packed,
                                 hipStream_t s);
hipError_t launch_rows4_unpack(const ql_rows4& d, int8_t* codes, void* scales, hipStream_t s);

// ------------------------------------------------------------- norms, turns ----

struct HeadsArgs {
  const void* x;
  int64_t xb, xr;
  const void* pos;
  int64_t pb;
  ql_heads_view y[3];  // q, k, v; in the gradient dq, dk, dv
  void* dx;
  int64_t db, dr;
  const void* gamma[2];
  const double* freqs;
  int heads[3];
  int B, L, D, n_axes, half[QL_MAX_AXES];  // half: pairs of an axis
  float eps;
  bool rms, halves, pos_f32, x_bf16, y_bf16, w_bf16;
  bool vec;       // rows of x and y can be read and written in vectors
  int tokens;     // tokens a workgroup turns at once (set by the launch)
  void* dgamma[2];
  float* part;    // [workgroups][2][D]
  int groups;     // workgroups of the gradient
};
// Workgroups of the gradient call (each has a row of partial sums).
int heads_grad_groups(int64_t tokens);
hipError_t launch_heads(const HeadsArgs& a, hipStream_t s);
hipError_t launch_heads_grad(const HeadsArgs& a, hipStream_t s);

// ---------------------------------------------------------------- attention ----

// Queries of the G = H / Hk heads that share a key head are rows of one matrix, row
// r = l * G + g, so shared heads need no care in the kernels: they read a key once for
// all of its rows, and the gradients of keys sum over all of them.
struct AttnArgs {
  ql_heads_view q, k, v, o, dout, dq, dk, dv;
  float* lse;    // [B, H, Lq]; forward: may be nullptr
  float* delta;  // [B, H, Lq]
  const int32_t* lens;
  const uint8_t* mask;
  int64_t mask_batch;
  int B, H, Hk, G, Lq, Lk, D, R;  // R = Lq * G
  int unit;      // neighbouring key heads that share an L2
  float scale, scale2;            // scale2 = scale * log2(e)
  int row_tiles, key_tiles, per_group;
  int splits;       // of the keys (forward), of the rows (dk and dv)
  float* part;      // forward [splits][B, H, Lq][D]; dk, dv: [workgroup][2][128 keys][D]
  float* part_lse;  // [splits][B, H, Lq], base 2
  bool bf16;
  bool near_keys;   // 128 rows of k and of v lie within 32-bit offsets
  bool near_rows;   // 32 rows of q and of dout lie evenly and within 32-bit offsets
};
struct AttnPlan {
  bool narrow;               // forward, fp32, few rows: waves share the keys
  int per_group;             // forward, few keys: tiles of rows of a workgroup, else 0
  int row_tiles, splits;          // forward
  int q_tiles, key_tiles, k_splits;  // gradient
  int64_t forward_bytes, grad_bytes;
};
AttnPlan attn_plan(const ql_attn& d);
hipError_t launch_attn(const AttnArgs& a, const AttnPlan& p, hipStream_t s);
hipError_t launch_attn_grad(const AttnArgs& a, const AttnPlan& p, hipStream_t s);

// One object file for each head size and type defines its own; DC = 16-channel blocks.
#define QL_ATTN_UNIT(T, DC)                                                        \
  hipError_t attn_forward_##T##_##DC(const AttnArgs& a, const AttnPlan& p, hipStream_t); \
  hipError_t attn_grad_##T##_##DC(const AttnArgs& a, const AttnPlan& p, hipStream_t);
#define QL_ATTN_UNITS(X) \
  X(f32, 2) X(f32, 4) X(f32, 5) X(f32, 6) X(f32, 8) X(f32, 10) \
  X(bf16, 2) X(bf16, 4) X(bf16, 5) X(bf16, 6) X(bf16, 8) X(bf16, 10)
#define QL_ATTN_DECL(T, DC) QL_ATTN_UNIT(T, DC)
QL_ATTN_UNITS(QL_ATTN_DECL)

}  // namespace ql
