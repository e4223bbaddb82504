// Host-side launchers of the fused layer, the expert products and the expert
// router.  Arguments are validated by the C ABI layer; each launcher returns
// hipGetLastError() after enqueueing its kernels on `stream`.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace awq {

// A stack of E packed weights of one shape (E = 1: a single layer).
struct PackedArgs {
  const uint32_t* qweight;
  const uint16_t* scales;
  const uint32_t* qzeros;  // NULL: symmetric
  int E, N, K, group_size;
};

// Y[r] = act(X[row(r)] W'_e^T + bias_e) [* the second half of the columns] +
// residual[r] for R rows; `offsets` NULL: one expert holds all R rows.
struct ProductArgs {
  const _Float16* x;
  int64_t ldx;
  int x_rows;                // rows of x
  const int* rows;           // NULL: row r of x; else row rows[r] / slots_per_row
  int slots_per_row;
  const int* offsets;        // [E + 1], or NULL
  int R;
  const _Float16* bias;      // [E][N], or NULL
  int activation;            // awq_activation
  bool gated;
  const _Float16* residual;  // [R][N_out] at stride ldr, or NULL
  int64_t ldr;
  _Float16* y;               // [R][N_out] at stride ldy
  int64_t ldy;
};

// The weighted sum over each token's slots: y[t] = sum_j weights[t][j] *
// (product row positions[t][j]) + residual[t].
struct CombineArgs {
  const int* positions;  // [T][top_k], negative: not routed
  const float* weights;  // [T][top_k]
  int T, top_k;
  const _Float16* residual;
  int64_t ldr;
  _Float16* y;
  int64_t ldy;
};

// Matrix-core tiles (awq_expert_tiles.hip): most rows of a tile, K split.  With
// `part` the raw sums (the bias in slice 0's) go to part[split][R][N].
struct TilePlan {
  int rows, splits, steps_per_split;
};
hipError_t launch_tiles(const PackedArgs& w, const ProductArgs& p, int gshift, const TilePlan& plan, float* part,
                        hipStream_t stream);

// Weight-stream tiles (awq_expert_stream.hip): most rows of a tile (16, 32, 64),
// waves along the weight rows and along K, K split across workgroups.
struct StreamPlan {
  int rows, cw, kw, splits;
};
hipError_t launch_stream(const PackedArgs& w, const ProductArgs& p, int gshift, const StreamPlan& plan, float* part,
                         hipStream_t stream);

// One row at a time (awq_fused_gemv.hip): R rows, each with its expert's whole
// weight; and T tokens' weighted sums.
hipError_t launch_fused_gemv(const PackedArgs& w, const ProductArgs& p, int gshift, hipStream_t stream);
hipError_t launch_combine_gemv(const PackedArgs& w, const ProductArgs& p, const CombineArgs& c, int gshift,
                               hipStream_t stream);

// A few rows (awq_fused_few.hip): tiles of at most 4 rows, or 8 (one layer); N * K < 2^32.
hipError_t launch_few(const PackedArgs& w, const ProductArgs& p, int gshift, int rows, float* part, hipStream_t stream);

size_t product_workspace_bytes(int R, int E, int N, int K, int group_size);
hipError_t launch_product(const PackedArgs& w, const ProductArgs& p, void* workspace, hipStream_t stream);

// `p` describes the product (x already sorted by expert, no gather, gate or
// residual); its y is not used.
size_t combine_workspace_bytes(int T, int top_k, int E, int N, int K, int group_size);
hipError_t launch_combine(const PackedArgs& w, const ProductArgs& p, const CombineArgs& c, void* workspace,
                          hipStream_t stream);

size_t route_workspace_bytes(int T, int E);
hipError_t launch_route(const void* logits, int ld, bool fp32, int T, int E, int top_k, bool renormalize, int* ids,
                        float* weights, int* offsets, int* rows, int* positions, void* workspace, hipStream_t stream);

}  // namespace awq
