// The 4-bit layer with its epilogue, and the same layer over rows grouped by
// expert:
//   Y[r] = act(X[row(r)] . W'_e^T + b_e) [* (X[row(r)] . U'_e^T + c_e)] + residual[r]
// with e the expert of row r (one expert for awq_linear_fused), and the
// weighted sum of such rows per token (awq_combine_experts).  A gated layer
// stores its gate rows W' first and the rows U' they multiply second, in one
// packed weight of N = 2 F rows.
#include "awq_epilogue.hpp"
#include "awq_launch_fused.hpp"

#include <math.h>

namespace awq {
namespace {

int log2_group(int g) { return g == 32 ? 5 : g == 64 ? 6 : g == 128 ? 7 : 8; }

// The two kernels below: a single wave per workgroup, four columns of one row
// per thread, so that a few rows spread over the chip and no thread divides (13 x
// 11008 -> 4096, K in 4: about 3 of 16.2 us are this launch).  Past kFinishRows
// rows a workgroup takes every kFinishRows-th.
constexpr int kFinish = 64, kFinishRows = 32768;

dim3 finish_grid(int columns, int rows) {
  return dim3((unsigned)((columns / 4 + kFinish - 1) / kFinish), (unsigned)(rows < kFinishRows ? rows : kFinishRows));
}

// part[row][n .. n + 3] summed over the K slices in order.
__device__ __forceinline__ float4_t slices_sum(const float* __restrict__ part, int splits, int64_t rows, int N,
                                               int64_t row, int n) {
  float4_t v = *reinterpret_cast<const float4_t*>(part + row * N + n);
#pragma unroll 4
  for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const float4_t*>(part + (s * rows + row) * N + n);
  return v;
}

// The rows that the experts' ranges hold: only their sums were written.
__device__ __forceinline__ int first_row(const ProductArgs& p) { return p.offsets ? max(p.offsets[0], 0) : 0; }
__device__ __forceinline__ int end_row(const ProductArgs& p, int E) { return p.offsets ? min(p.offsets[E], p.R) : p.R; }

// The epilogue of a product whose K was split.
__global__ __launch_bounds__(kFinish) void finish_kernel(const float* __restrict__ part, int splits, PackedArgs w,
                                                         ProductArgs p) {
  const int width = p.gated ? w.N >> 1 : w.N, n = (blockIdx.x * kFinish + threadIdx.x) * 4;
  if (n >= width) return;
  const int rows = end_row(p, w.E);
  for (int row = first_row(p) + blockIdx.y; row < rows; row += gridDim.y) {
    float4_t v = slices_sum(part, splits, p.R, w.N, row, n);
    float4_t up = {1.f, 1.f, 1.f, 1.f};
    if (p.gated) up = slices_sum(part, splits, p.R, w.N, row, width + n);
    half4_t out;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float o = activate(v[k], p.activation);
      if (p.gated) o *= up[k];
      if (p.residual) o += (float)p.residual[row * p.ldr + n + k];
      out[k] = (_Float16)o;
    }
    *reinterpret_cast<half4_t*>(p.y + row * p.ldy + n) = out;
  }
}

// y[t] = sum over the slots j, in order, of weights[t][j] * part[positions[t][j]]
// + residual[t], over the slots whose rows the experts' ranges hold.
__global__ __launch_bounds__(kFinish) void combine_kernel(const float* __restrict__ part, int splits, PackedArgs w,
                                                          ProductArgs p, CombineArgs c) {
  const int n = (blockIdx.x * kFinish + threadIdx.x) * 4, N = w.N;
  if (n >= N) return;
  const int first = first_row(p), end = end_row(p, w.E);
  for (int t = blockIdx.y; t < c.T; t += gridDim.y) {
    float4_t sum = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < c.top_k; ++j) {
      const int at = c.positions[(int64_t)t * c.top_k + j];
      if (at < first || at >= end) continue;
      sum += c.weights[(int64_t)t * c.top_k + j] * slices_sum(part, splits, p.R, N, at, n);
    }
    half4_t out;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (c.residual) sum[k] += (float)c.residual[t * c.ldr + n + k];
      out[k] = (_Float16)sum[k];
    }
    *reinterpret_cast<half4_t*>(c.y + t * c.ldy + n) = out;
  }
}

// How a product runs: one row or a few at a time, the weight stream, or the
// matrix-core tiles.
struct Plan {
  enum Kind { kFew, kStream, kTiles } kind;
  int few_rows;
  StreamPlan stream;
  TilePlan tile;
  int splits() const { return kind == kStream ? stream.splits : kind == kTiles ? tile.splits : 1; }
};

// One row per workgroup set: a single token, or so few rows that experts with
// two are rare (their weights are then read twice, the second time from L2).  us,
// one row at a time / tiles of 4 rows, at R = E / 2: 2 tokens x 2 of 8, 4096 ->
// 22016 gated: 34 / 40; 2 x 4 of 16, 4096 -> 8192: 27 / 30; 8 x 8 of 128, 2048 ->
// 1536 gated: 22 / 24.  At R = E: 4 x 2 of 8: 60.5 / 58.9; 4 x 4 of 16: 45.1 / 43.6.
bool one_row_each(int R, int E) { return R == 1 || 2 * R <= E; }

// Tiles of a few rows: up to 8 tokens of one layer, up to 3 rows for every two
// experts.  us, few rows / the best of the weight stream: 8 x 4096 -> 4096: 6.2 /
// 9.1; 8 x 11008 -> 4096: 12.8 / 14.5; 8 x 4096 -> 11008: 12.1 / 10.9 (they hold 8
// rows at most: 9 take two).  Experts at R = E: 16 x 8 of 128, 768 -> 2048
// combined: 27.7 / 30.2; 4 x 4 of 16, 4096 -> 8192: 43.6 / 45.6; at 1.5 E: 16 x 6 of 64, 2048 -> 2816
// gated: 36.1 / 36.4; at 2 E: 8 x 2 of 8, 11008 -> 4096 combined: 58.2 / 44.1;
// 32 x 8 of 128, 2048 -> 1536 gated: 49.4 / 44.6.
bool few_rows_each(int R, int E) { return E == 0 ? R <= 8 : 2 * R <= 3 * E; }

// Past that a time model chooses among five weight-stream variants and two tile
// heights, each with K whole or split across workgroups.  Each of 256 compute
// units takes its share of the workgroups, one at a time or two at once where two
// fit its LDS; a workgroup takes `begin` us and `one` (two at once: `two`) for each
// of its stages or steps; partial sums cost a launch (4 us) and are written and
// read at 5.5 TB/s.  The constants are fitted to 1687 measured plans of 177 shapes
// in groups of 128 (1-256 rows of nine layers, N and K from 768 to 28672; 2-256
// tokens through 2 of 8, 4 of 16, 6 of 64 and 8 of 128 experts, combined and not;
// 300-2048 rows on tiles): half the plans are within 7%.  The choices are on
// average 1% above the best plan measured, over those and 75 shapes that are not
// among them (300-2048 rows); worst: 500 tokens x 6 of 64, 1408 -> 2048 combined, 83 / 62.
// Two sides (us, the choice / another):
//   16 x 4096 -> 4096: 16 rows, 2 x 2 waves, K in 4: 9.6-9.8 / whole: 11.0; 2 x 4 waves: 9.2
//   13 x 11008 -> 4096: 16 rows, 2 x 4 waves, K in 4: 16.2 / 2 x 4, whole: 23
//   64 x 4096 -> 4096: 16 rows, 2 x 4 waves: 9.8 / 32 rows, 4 x 2, K in 4: 12.7
//   48 tokens x 6 of 64, 2048 -> 2816 gated: 32 rows, 4 x 1: 46.6 / 16 rows, 2 x 2: 54
//   61 x 4096 -> 11008: 32 rows, 4 x 2: 18 / 4 x 1: 20.9; 64 rows, K in 2: 22.7
//   64 x 8192 -> 28672: 64 rows, 4 x 1: 56.6 / 32 rows, 4 x 1: 58.5, 4 x 2: 62.9
//   100 x 8192 -> 28672: 64 rows, 4 x 1: 85-87 / 32 rows, 4 x 1: 104
//   200 x 8192 -> 28672: tiles of 128 rows: 128 / stream, 64 rows: 160
//   512 x 4096 -> 11008: tiles of 128 rows: 70 / in 2: 77; 64 rows: 78; stream: 69
//   700 x 4096 -> 11008: tiles of 64 rows: 81-89 / 128 rows: 101-106
//   512 x 11008 -> 4096: tiles of 128 rows in 4: 63 / whole: 167; 64 rows, whole: 131
//   1000 tokens x 2 of 8, 11008 -> 4096 combined: tiles, K in 3: 241 / whole: 307-320
struct StreamKind {
  int rows, cw, kw;
  bool pairs;  // two workgroups fit a compute unit
  double one, two, begin;
};
constexpr StreamKind kStreamKinds[] = {{16, 2, 2, true, 1.0, 1.6, 2.7},
                                       {16, 2, 4, false, 1.7, 0.0, 2.7},
                                       {32, 4, 1, true, 1.0, 1.6, 2.6},
                                       {32, 4, 2, false, 1.6, 0.0, 2.9},
                                       {64, 4, 1, true, 0.74, 1.2, 3.1}};

// The most loaded unit's time with `count` workgroups of `steps` steps.
double unit_us(double count, int steps, bool pairs, double one, double two, double begin) {
  const int each = (int)ceil(count / 256.0);
  if (!pairs) return each * (steps * one + begin);
  return (each / 2) * (steps * two + begin) + (each % 2) * (steps * one + begin);
}

// `summed`: the products are partial sums in any case (combining).
Plan plan_by_time(int R, int experts, int N, int K, int group_size, bool summed) {
  const double each = (double)R / experts;
  // groups of 32 apply a scale every two matrix instructions
  const double slow = group_size == 32 ? 1.3 : 1.0;
  // ragged experts end in half a tile each on average
  auto row_tiles_of = [&](int rows) {
    const double n = each / rows + 0.5;
    return experts == 1 ? (double)((R + rows - 1) / rows) : experts * (n < 1 ? 1 : n);
  };
  auto sums_us = [&](int splits) { return splits > 1 || summed ? 4.0 + splits * (double)R * N * 8 / 5.5e6 : 0.0; };
  Plan best{Plan::kTiles, 0, {}, TilePlan{64, 1, (K + 63) / 64}};
  double best_us = 1e300;
  // (the stream addresses an expert's packed words with 31 bits)
  if ((int64_t)N * K < ((int64_t)1 << 32)) {
    for (const StreamKind& v : kStreamKinds) {
      const int channels = (v.rows <= 32 ? 256 : 128) * v.kw, stages = (K + channels - 1) / channels;
      const int columns = (N + 32 * v.cw - 1) / (32 * v.cw);
      const double tiles = row_tiles_of(v.rows) * columns;
      // (a launch holds less than 2^32 threads; with half of that most tiles there can be)
      if ((double)((R + v.rows - 1) / v.rows + experts) * columns * (64 * v.cw * v.kw) >= 2147483648.0) continue;
      for (int s = 1; s <= 8 && s <= stages; ++s) {
        const int per = (stages + s - 1) / s, splits = (stages + per - 1) / per;
        // no empty slice, and none of a single stage: its loads would run beside nothing
        if (splits != s || (s > 1 && per < 2)) continue;
        const double us =
            unit_us(tiles * splits, per, v.pairs, slow * v.one, slow * v.two, v.begin) + sums_us(splits);
        if (us < best_us) best_us = us, best = Plan{Plan::kStream, 0, StreamPlan{v.rows, v.cw, v.kw, splits}, {}};
      }
    }
  }
  const int steps = (K + 63) / 64, columns = (N + 255) / 256;
  for (int rows : {group_size == 32 ? 96 : 128, 64}) {
    if (each <= 32 && best.kind == Plan::kStream) break;  // a tile has 64 rows at least to multiply
    const double tiles = row_tiles_of(rows), mean = R / tiles / 32;
    const double height = mean < 2 ? 2 : experts == 1 ? ceil(mean) : mean;
    const double one = slow * (0.51 + 0.107 * height), two = slow * (0.73 + 0.245 * height);
    for (int s = 1; s <= 16 && s <= steps; ++s) {
      // (slices of an even number of steps: no group of 128 channels is cut)
      const int per = s == 1 ? steps : ((steps + s - 1) / s + 1) & ~1, splits = (steps + per - 1) / per;
      if (splits != s) continue;
      const double us = unit_us(tiles * columns * splits, per, true, one, two, 5.5) + sums_us(splits);
      if (us < best_us) best_us = us, best = Plan{Plan::kTiles, 0, {}, TilePlan{rows, splits, per}};
    }
  }
  return best;
}

// E = 0: one expert, R rows known to the host.  Experts' counts live on the
// device: the plan is for their average.
Plan plan_product(int R, int E, int N, int K, int group_size, bool summed) {
  // (an expert's packed words are addressed with 31 bits there, too)
  if (few_rows_each(R, E) && (int64_t)N * K < ((int64_t)1 << 32))
    return Plan{Plan::kFew, E == 0 && R > 4 ? 8 : 4, {}, {}};
  return plan_by_time(R, E == 0 ? 1 : E < R ? E : R, N, K, group_size, summed);
}

size_t part_bytes(const Plan& plan, int R, int N) {
  return gemm_counter_bytes() + (size_t)plan.splits() * R * N * 4;
}

float* part_of(void* workspace) {
  return reinterpret_cast<float*>(static_cast<char*>(workspace) + gemm_counter_bytes());
}

hipError_t launch_planned(const PackedArgs& w, const ProductArgs& p, const Plan& plan, float* part,
                          hipStream_t stream) {
  const int gs = log2_group(w.group_size);
  switch (plan.kind) {
    case Plan::kFew: return launch_few(w, p, gs, plan.few_rows, part, stream);
    case Plan::kStream: return launch_stream(w, p, gs, plan.stream, part, stream);
    default: return launch_tiles(w, p, gs, plan.tile, part, stream);
  }
}

}  // namespace

size_t product_workspace_bytes(int R, int E, int N, int K, int group_size) {
  if (one_row_each(R, E)) return 0;
  const Plan plan = plan_product(R, E, N, K, group_size, false);
  return plan.splits() > 1 ? part_bytes(plan, R, N) : 0;
}

hipError_t launch_product(const PackedArgs& w, const ProductArgs& p, void* workspace, hipStream_t stream) {
  if (one_row_each(p.R, p.offsets ? w.E : 0)) return launch_fused_gemv(w, p, log2_group(w.group_size), stream);
  const Plan plan = plan_product(p.R, p.offsets ? w.E : 0, w.N, w.K, w.group_size, false);
  if (plan.splits() <= 1) return launch_planned(w, p, plan, nullptr, stream);
  float* part = part_of(workspace);
  const hipError_t e = launch_planned(w, p, plan, part, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(finish_kernel, finish_grid(p.gated ? w.N / 2 : w.N, p.R), dim3(kFinish), 0, stream, part,
                     plan.splits(), w, p);
  return hipGetLastError();
}

size_t combine_workspace_bytes(int T, int top_k, int E, int N, int K, int group_size) {
  if (one_row_each(T * top_k, E)) return 0;
  return part_bytes(plan_product(T * top_k, E, N, K, group_size, true), T * top_k, N);
}

hipError_t launch_combine(const PackedArgs& w, const ProductArgs& p, const CombineArgs& c, void* workspace,
                          hipStream_t stream) {
  if (one_row_each(p.R, w.E)) return launch_combine_gemv(w, p, c, log2_group(w.group_size), stream);
  const Plan plan = plan_product(p.R, w.E, w.N, w.K, w.group_size, true);
  float* part = part_of(workspace);
  const hipError_t e = launch_planned(w, p, plan, part, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(combine_kernel, finish_grid(w.N, c.T), dim3(kFinish), 0, stream, part, plan.splits(), w, p, c);
  return hipGetLastError();
}

}  // namespace awq
