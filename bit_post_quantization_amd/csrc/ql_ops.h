// Internal interface between the C ABI of the operators beside the layer
// (qlinear_ops.cpp) and their kernels (k_lora.hip, k_norm.hip, k_clip.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qlinear.h"

namespace ql {

// ---------------------------------------------------------------- adapters ----

// Rows of a batch split into requests: request i owns rows [off[i], off[i+1])
// and runs adapter ids[i] (none where that is outside [0, n_adapters)). All of
// it is device data, so kernels clamp what they read.
struct Requests {
  const int32_t* off;
  const int32_t* ids;
  int n;
  int rows;        // rows that the offsets partition
  int n_adapters;
};

// part[split][row][j] = scale_a * sum over the split's columns n of
// dY[row][n] * B_a[n][j], for the rows of every request with an adapter.
struct DsArgs {
  const float* dY;    // [rows, N], row stride ldy elements
  int64_t ldy;
  const void* B;      // [n_adapters, N, rank]
  const float* scales;// per adapter, or nullptr (1)
  const int32_t* ranks;
  Requests q;
  int N, rank;
  int splits, split_len;  // columns of a split, a multiple of kDsStep
  float* part;        // [splits][rows][rank]; nullptr: not wanted
  bool tall;
  bool vec;           // 16-byte pieces of dY (set by the launch)
};
constexpr int kDsStep = 32;

// Y[row][n] = base[row][n] + scale_a * sum_j S[row][j] * B_a[n][j] with
// S = X A_a^T, combined over the row's two halves when guided.
struct ForwardArgs {
  const void* X;      // [rows * halves, K], row stride ldx elements
  int64_t ldx;
  const void* A;      // [n_adapters, rank, K]
  const void* B;      // [n_adapters, N, rank]
  const float* scales;
  const int32_t* ranks;
  Requests q;
  int N, K, rank, halves;
  float w;            // guidance weight (halves == 2)
  const float* base;  // nullptr: zero
  float* Y;
  int64_t ldb, ldy;
  float* S;           // nullptr, or [rows * halves, rank]
  void* ws;           // lora_forward_ws() bytes
  int shares;         // workgroups of one tile of rows (set by the launch)
  bool x_bf16, w_bf16;
};

// Row ranges s = 0 .. splits-1 of row_len rows each. For every range and the
// requests i in it, slot s + i of `out` receives the sum over the common rows (those
// of neighbouring requests of one adapter together, in the last one's slot)
// of Q[row][j] * P[row][d] ([j][d] for dA, [d][j] for dB);
// slot_id[s + i] says which adapter it belongs to (-1: nothing was written).
// With dX, dX[row][d] = sum_j Q[row][j] * A_a[j][d] too (zero for rows without
// an adapter).
struct OuterArgs {
  const void* P;      // [rows, D]
  int64_t ldp;
  const float* part;  // Q: [q_splits][rows][rank]
  int q_splits;
  const void* A;      // [n_adapters, rank, D] (dX)
  const int32_t* ranks;
  Requests q;
  int D, rank;
  void* dX;           // nullptr: none; else of P's type
  int64_t lddx;
  float* out;         // [slots][D * rank]; nullptr: this side is not wanted
  int32_t* slot_id;   // [slots]
  int splits, row_len;
  bool p_bf16, w_bf16;
  int chunks;         // set by the launch, as are the next three
  bool p_vec, q_vec, dx_vec;  // vectors of P, Q and dX are aligned
};

// dW[a][e] = scale_a * sum over the slots of adapter a of part[slot][e].
struct SlotSumArgs {
  const float* part;
  const int32_t* slot_id;
  int slots, n_adapters, D, rank;
  const float* scales;  // nullptr: 1
  const int32_t* ranks;
  void* out;
  bool w_bf16, transposed;
};

// Workspace of a forward call with `rows` output rows.
int64_t lora_forward_ws(int rows, int n_req, int N, int rank, bool w_bf16);
// Whether the call's launches stay within the grid's limit.
bool lora_fits(int rows, int n_req, int N, bool grad);
hipError_t launch_lora_forward(const ForwardArgs& a, hipStream_t s);
bool lora_ds_tall(int rows, int n_req);
int lora_ds_splits(int rows, int n_req, int N);
// Row ranges of dA's and dB's sums.
int lora_x_splits(int rows, int K);
int lora_y_splits(int rows, int n_req, int N);
// dS and dB.
hipError_t launch_lora_grad_y(const DsArgs& d, const OuterArgs& y, hipStream_t s);
// dA and dX.
hipError_t launch_lora_grad_x(const OuterArgs& x, hipStream_t s);
// The sums of both sides; one without `out` is left out.
hipError_t launch_lora_slot_sum(const SlotSumArgs& p, const SlotSumArgs& q, hipStream_t s);

// -------------------------------------------------------------- group norm ----

struct NormArgs {
  const void* x;
  int64_t xb, xr;     // element strides of an image and of a position
  const void* dy;     // gradient only
  int64_t dyb, dyr;
  void* y;            // y, or dx
  int64_t yb, yr;
  const void* gamma;
  const void* beta;
  int B, L, C, G;
  float eps;
  int act;
  float* mean;        // [B, G]: out (may be nullptr) / in (gradient)
  float* rstd;
  void* dgamma;
  void* dbeta;
  void* ws;
  bool x_bf16, w_bf16;
};
// es: bytes of an element.
int64_t norm_ws_bytes(int B, int L, int C, int G, int es, bool grad);
hipError_t launch_group_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_group_norm_grad(const NormArgs& a, hipStream_t s);

// ---------------------------------------------------------------- clipping ----

hipError_t launch_grad_norm(const ql_grad* table, int n, int64_t units, double* partials,
                            hipStream_t s);
hipError_t launch_grad_clip(const ql_grad* table, int n, int64_t units, const double* partials,
                            float max_norm, float* norm, hipStream_t s);

}  // namespace ql
