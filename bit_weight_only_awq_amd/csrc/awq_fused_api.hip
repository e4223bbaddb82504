// C ABI of the fused layer, the expert router and the expert products:
// argument validation, then the launches on the caller's stream.  The
// contract of every entry point is in include/awq.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/awq.h"
#include "awq_launch.hpp"
#include "awq_launch_fused.hpp"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }  // offsets: read one by one

constexpr int32_t kMaxDim = 1 << 21;
constexpr int32_t kMaxRows = 1 << 24;     // tokens, slots: keeps launch grids and row tiles in 32 bits
constexpr int32_t kMaxExperts = 1024;
constexpr int32_t kMaxTopK = 64;

// A row stride: at least the row, rows 16-byte aligned, a tile of 256 rows
// within the kernels' 32-bit byte offsets.
bool stride_ok(int32_t ld, int32_t row) { return ld >= row && ld <= kMaxDim && (ld & 7) == 0; }

// Gathered rows of x are addressed with 31-bit byte offsets from its first.
bool gather_ok(int32_t rows, int32_t ld) { return (int64_t)rows * ld < ((int64_t)1 << 30); }

// The weight's shape and pointers, the epilogue's options and pointers: what
// every product checks.
int check_product(int32_t N, int32_t K, int32_t group_size, int32_t zero_point, const uint32_t* qweight,
                  const void* scales, const uint32_t* qzeros, const void* bias, int32_t activation, int32_t gated,
                  const void* residual, int32_t ldr, const void* x, int32_t ldx, const void* y, int32_t ldy) {
  if (group_size != 32 && group_size != 64 && group_size != 128 && group_size != 256) return AWQ_ERR_GROUP;
  if (N < 1 || K < 1 || (N & (gated ? 15 : 7)) != 0 || N > kMaxDim || K > kMaxDim) return AWQ_ERR_SHAPE;
  if (K % group_size != 0) return AWQ_ERR_GROUP;
  const int32_t width = gated ? N / 2 : N;
  if (!stride_ok(ldx, K) || !stride_ok(ldy, width) || (residual && !stride_ok(ldr, width))) return AWQ_ERR_SHAPE;
  if (activation < AWQ_ACT_NONE || activation > AWQ_ACT_GELU_TANH) return AWQ_ERR_OPTION;
  if (!x || !y || !qweight || !scales || (zero_point && !qzeros)) return AWQ_ERR_NULL;
  if (!aligned16(x) || !aligned16(y) || !aligned16(qweight) || !aligned16(scales) ||
      (zero_point && !aligned16(qzeros)) || !aligned16(bias) || !aligned16(residual))
    return AWQ_ERR_ALIGN;
  return AWQ_OK;
}

int check_workspace(const void* workspace, size_t have, size_t need) {
  if (have < need) return AWQ_ERR_WORKSPACE;
  if (need > 0 && !workspace) return AWQ_ERR_NULL;
  return need > 0 && !aligned16(workspace) ? AWQ_ERR_ALIGN : AWQ_OK;
}

bool shape_known(int32_t N, int32_t K, int32_t group_size, int32_t gated) {
  return (group_size == 32 || group_size == 64 || group_size == 128 || group_size == 256) && N >= 1 && K >= 1 &&
         (N & (gated ? 15 : 7)) == 0 && N <= kMaxDim && K <= kMaxDim && K % group_size == 0;
}

int from_hip(hipError_t e) { return e == hipSuccess ? AWQ_OK : AWQ_ERR_HIP; }

awq::PackedArgs packed(const uint32_t* qweight, const void* scales, const uint32_t* qzeros, int32_t zero_point,
                       int32_t E, int32_t N, int32_t K, int32_t group_size) {
  return awq::PackedArgs{qweight, static_cast<const uint16_t*>(scales), zero_point ? qzeros : nullptr, E, N, K,
                         group_size};
}

const _Float16* halves(const void* p) { return static_cast<const _Float16*>(p); }

}  // namespace

extern "C" {

size_t awq_linear_fused_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t group_size, int32_t gated) {
  if (M < 1 || M > kMaxRows || !shape_known(N, K, group_size, gated)) return 0;
  return awq::product_workspace_bytes(M, 0, N, K, group_size);
}

int awq_linear_fused(const void* x, int32_t ldx, const uint32_t* qweight, const void* scales, const uint32_t* qzeros,
                     const void* bias, int32_t activation, int32_t gated, const void* residual, int32_t ldr, void* y,
                     int32_t ldy, int32_t M, int32_t N, int32_t K, int32_t group_size, int32_t zero_point,
                     void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_product(N, K, group_size, zero_point, qweight, scales, qzeros, bias, activation, gated, residual, ldr,
                         x, ldx, y, ldy);
  if (st != AWQ_OK) return st;
  if (M < 1 || M > kMaxRows) return AWQ_ERR_SHAPE;
  st = check_workspace(workspace, workspace_bytes,
                       awq_linear_fused_workspace_bytes(M, N, K, group_size, gated));
  if (st != AWQ_OK) return st;
  awq::ProductArgs p{halves(x), ldx,  M, nullptr, 1, nullptr, M, halves(bias), activation, gated != 0, halves(residual),
                     ldr, static_cast<_Float16*>(y), ldy};
  return from_hip(awq::launch_product(packed(qweight, scales, qzeros, zero_point, 1, N, K, group_size), p, workspace,
                                      static_cast<hipStream_t>(stream)));
}

size_t awq_route_experts_workspace_bytes(int32_t T, int32_t E) {
  if (T < 1 || T > kMaxRows || E < 1 || E > kMaxExperts) return 0;
  return awq::route_workspace_bytes(T, E);
}

int awq_route_experts(const void* logits, int32_t ld, int32_t fp32_logits, int32_t T, int32_t E, int32_t top_k,
                      int32_t renormalize, int32_t* ids, float* weights, int32_t* offsets, int32_t* rows,
                      int32_t* positions, void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 1 || T > kMaxRows || E < 1 || E > kMaxExperts || ld < E || ld > kMaxDim) return AWQ_ERR_SHAPE;
  if (top_k < 1 || top_k > E || top_k > kMaxTopK) return AWQ_ERR_OPTION;
  if ((int64_t)T * top_k > kMaxRows) return AWQ_ERR_SHAPE;
  if (!logits || !ids || !weights || !offsets || !rows || !positions) return AWQ_ERR_NULL;
  if (!aligned16(logits) || !aligned16(ids) || !aligned16(weights) || !aligned16(offsets) || !aligned16(rows) ||
      !aligned16(positions))
    return AWQ_ERR_ALIGN;
  const int st = check_workspace(workspace, workspace_bytes, awq_route_experts_workspace_bytes(T, E));
  if (st != AWQ_OK) return st;
  return from_hip(awq::launch_route(logits, ld, fp32_logits != 0, T, E, top_k, renormalize != 0, ids, weights, offsets,
                                    rows, positions, workspace, static_cast<hipStream_t>(stream)));
}

size_t awq_linear_experts_workspace_bytes(int32_t R, int32_t E, int32_t N, int32_t K, int32_t group_size,
                                          int32_t gated) {
  if (R < 1 || R > kMaxRows || E < 1 || E > kMaxExperts || !shape_known(N, K, group_size, gated)) return 0;
  return awq::product_workspace_bytes(R, E, N, K, group_size);
}

int awq_linear_experts(const void* x, int32_t ldx, int32_t x_rows, const int32_t* rows, int32_t slots_per_row,
                       const int32_t* offsets, int32_t R, int32_t E, const uint32_t* qweight, const void* scales,
                       const uint32_t* qzeros, const void* bias, int32_t activation, int32_t gated, void* y,
                       int32_t ldy, int32_t N, int32_t K, int32_t group_size, int32_t zero_point, void* workspace,
                       size_t workspace_bytes, void* stream) {
  int st = check_product(N, K, group_size, zero_point, qweight, scales, qzeros, bias, activation, gated, nullptr, 0, x,
                         ldx, y, ldy);
  if (st != AWQ_OK) return st;
  if (R < 1 || R > kMaxRows || E < 1 || E > kMaxExperts || x_rows < 1 || x_rows > kMaxRows ||
      (rows ? !gather_ok(x_rows, ldx) : x_rows < R))
    return AWQ_ERR_SHAPE;
  if (rows && slots_per_row < 1) return AWQ_ERR_OPTION;
  if (!offsets) return AWQ_ERR_NULL;
  if (!aligned4(offsets) || !aligned16(rows)) return AWQ_ERR_ALIGN;
  st = check_workspace(workspace, workspace_bytes,
                       awq_linear_experts_workspace_bytes(R, E, N, K, group_size, gated));
  if (st != AWQ_OK) return st;
  awq::ProductArgs p{halves(x), ldx, x_rows, rows, slots_per_row, offsets, R, halves(bias), activation, gated != 0,
                     nullptr, 0, static_cast<_Float16*>(y), ldy};
  return from_hip(awq::launch_product(packed(qweight, scales, qzeros, zero_point, E, N, K, group_size), p, workspace,
                                      static_cast<hipStream_t>(stream)));
}

size_t awq_combine_experts_workspace_bytes(int32_t T, int32_t top_k, int32_t E, int32_t N, int32_t K,
                                           int32_t group_size) {
  if (T < 1 || top_k < 1 || (int64_t)T * top_k > kMaxRows || E < 1 || E > kMaxExperts ||
      !shape_known(N, K, group_size, 0))
    return 0;
  return awq::combine_workspace_bytes(T, top_k, E, N, K, group_size);
}

int awq_combine_experts(const void* x, int32_t ldx, const int32_t* offsets, const int32_t* positions,
                        const float* weights, int32_t T, int32_t top_k, int32_t E, const uint32_t* qweight,
                        const void* scales, const uint32_t* qzeros, const void* bias, const void* residual,
                        int32_t ldr, void* y, int32_t ldy, int32_t N, int32_t K, int32_t group_size,
                        int32_t zero_point, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_product(N, K, group_size, zero_point, qweight, scales, qzeros, bias, AWQ_ACT_NONE, 0, residual, ldr,
                         x, ldx, y, ldy);
  if (st != AWQ_OK) return st;
  if (T < 1 || E < 1 || E > kMaxExperts) return AWQ_ERR_SHAPE;
  if (top_k < 1 || top_k > E || top_k > kMaxTopK) return AWQ_ERR_OPTION;
  if ((int64_t)T * top_k > kMaxRows) return AWQ_ERR_SHAPE;
  if (!offsets || !positions || !weights) return AWQ_ERR_NULL;
  if (!aligned4(offsets) || !aligned16(positions) || !aligned16(weights)) return AWQ_ERR_ALIGN;
  st = check_workspace(workspace, workspace_bytes,
                       awq_combine_experts_workspace_bytes(T, top_k, E, N, K, group_size));
  if (st != AWQ_OK) return st;
  const int R = T * top_k;
  awq::ProductArgs p{halves(x), ldx, R, nullptr, 1, offsets, R, halves(bias), AWQ_ACT_NONE, false, nullptr, 0, nullptr,
                     0};
  awq::CombineArgs c{positions, weights, T, top_k, halves(residual), ldr, static_cast<_Float16*>(y), ldy};
  return from_hip(awq::launch_combine(packed(qweight, scales, qzeros, zero_point, E, N, K, group_size), p, c,
                                      workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
