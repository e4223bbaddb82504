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
// per thread, so that a few rows spread over the chip and no thread divides (of
// 12.2 us for 61 x 4096 -> 4096, K in 2, 2.4 are this launch).  Past kFinishRows
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

// How a product runs, by the rows per expert (on average: the host does not
// know the counts): a few, the weight stream, or the matrix cores.
struct Plan {
  enum Kind { kFew, kStream, kTiles } kind;
  int few_rows;
  StreamPlan stream;
  TilePlan tile;
  int splits() const { return kind == kStream ? stream.splits : kind == kTiles ? tile.splits : 1; }
};

// One row per workgroup set: a single token, or so few rows that experts with
// two are rare (their weights are then read twice, the second time from L2).
bool one_row_each(int R, int E) { return R == 1 || 2 * R <= E; }

// Tile height and K split of the matrix-core tiles, from a time model: each of 256
// compute units takes its share of the tiles (256 weight rows each, gated or not),
// two at a time.  A 64-channel step of one tile takes 0.55 us + 0.115 per 32 rows
// (128 rows: 1.01, 64: 0.78), of two tiles at once 0.7 + 0.25 (1.7, 1.2), 1.3 times
// that in groups of 32; 5 us begin and end a tile; partial sums are written and read at 5.5 TB/s and
// cost a launch (5 us).  us of the choice / of others, groups of 128:
//   512 x 4096 -> 11008: 128 rows: 69.7 / in 2: 77.5; 64 rows: 78.6
//   700 x 4096 -> 11008: 64 rows: 87.5 / 128 rows: 105.5 (258 tiles: two units have two)
//   512 x 11008 -> 4096: 128 rows in 4: 65.8 / in 3: 71.8, unsplit: 167; 64 rows: 131
//   1024 x 11008 -> 4096: 128 rows in 2: 109.1 / unsplit: 167, in 4: 113.1
//   1000 tokens x 2 of 8, 11008 -> 4096 combined: in 3: 251 / unsplit: 320, in 2: 257
//   2000 tokens x 6 of 64, 2048 -> 2816 gated: 196 / in 2: 291; 64 rows: 232
// (20 shapes: at most 4% above the best of seven plans.)  `summed`: the
// products are partial sums in any case (combining).
TilePlan plan_tiles(int R, int experts, int N, int K, int group_size, bool summed) {
  const int steps = (K + 63) / 64, columns = (N + 255) / 256;
  constexpr double kUnits = 256;
  const double slow = group_size == 32 ? 1.3 : 1.0;
  TilePlan best{64, 1, steps};
  double best_us = 1e300;
  for (int rows : {group_size == 32 ? 96 : 128, 64}) {
    // ragged experts end in half a tile each on average
    const double tiles = experts == 1 ? (R + rows - 1) / rows : experts * ((double)R / experts / rows + 0.5);
    const double mean = R / tiles / 32, height = experts == 1 ? ceil(mean) : mean < 1 ? 1 : mean;
    const double one = slow * (0.55 + 0.115 * height), two = slow * (0.7 + 0.25 * height);
    for (int s = 1; s <= 16 && s <= steps; ++s) {
      // (slices of an even number of steps: no group of 128 channels is cut)
      const int per = s == 1 ? steps : ((steps + s - 1) / s + 1) & ~1, splits = (steps + per - 1) / per;
      const int64_t each = (int64_t)ceil(tiles * columns * splits / kUnits);
      const double us = (each / 2) * (per * two + 5.0) + (each % 2) * (per * one + 5.0) +
                        (splits > 1 || summed ? splits * (double)R * N * 8 / 5.5e6 + 5.0 : 0.0);
      if (us < best_us) best_us = us, best = TilePlan{rows, splits, per};
    }
  }
  return best;
}

// Weight-stream tiles, by how many there are.  Many (c: 128-row columns times
// row tiles): 4 waves side by side.  Fewer: the waves of a workgroup split K, and
// then the workgroups do, until about 256 of them run.  us on the 7B shapes,
// the variant chosen / the one on the other side of the rule:
//   13 x 11008 -> 4096: 2 x 2 waves, K in 4: 14.9 / 2 x 4 waves, no split: 23.0
//   16 x 4096 -> 4096: 2 x 4: 9.1 / 4 x 1: 16.8;  16 x 4096 -> 11008: 11.6 / 17.9
//   16 x 4096 -> 32768: 2 x 2: 21.7 / 4 x 1 with 32 rows: 22.9 (with 16 rows: 22.3)
//   16 tokens x 2 of 8, 11008 -> 4096: 2 x 2: 47.2 / 4 x 1 with 32 rows: 54.4
//   48 tokens x 6 of 64, 2048 -> 2816: 4 x 1 with 32 rows: 46.1 / 2 x 2: 54.0
// (4 x 1 waves take tiles of 32 rows however few there are: an expert with 17 is
// then read once, and 96 tokens x 6 of 64 take 51.6 us against 57.0 with 16.)
//   61 x 4096 -> 11008 (32-row tiles): 4 x 2: 17.9 / 4 x 1: 20.8; 64 rows: 22.2
//   100 x 4096 -> 4096: 4 x 2, K in 2: 14.0 / 4 x 1: 27
//   200 x 4096 -> 11008: 4 x 1: 42.5 / 4 x 2: 46.5
StreamPlan plan_stream(int R, int experts, int N, int K) {
  const double each = (double)R / experts;
  auto plan = [&](int rows, int cw, int kw, int splits) {
    // no empty slice: every slice but the last has the same number of stages
    const int channels = (rows <= 32 ? 256 : 128) * kw, stages = (K + channels - 1) / channels;
    if (splits > stages / 2) splits = stages / 2;
    if (splits < 1) splits = 1;
    const int per = (stages + splits - 1) / splits;
    return StreamPlan{rows, cw, kw, (stages + per - 1) / per};
  };
  const int c64 = experts * ((N + 63) / 64);
  if (each <= (experts == 1 ? 16 : 10) || (experts == 1 && R <= 32 && K <= 6144 && 2 * c64 <= 160)) {
    const int c = each <= 16 ? c64 : 2 * c64;
    if (c >= 768) return plan(32, 4, 1, 1);
    if (c >= 224) return plan(16, 2, 2, 1);
    if (c >= 96 || K <= 6144) return plan(16, 2, 4, 1);
    return plan(16, 2, 2, c >= 64 ? 4 : 8);
  }
  if (experts > 1 && each > 40) return plan(64, 4, 1, 1);
  const double tiles = experts == 1 ? (R + 31) / 32 : experts * (each / 32 + 0.5);
  const double c = tiles * ((N + 127) / 128);
  if (c >= 320) return plan(32, 4, 1, 1);
  if (c >= 160) return plan(32, 4, 2, 1);
  return plan(32, 4, 2, c > 128 ? 1 : c > 80 ? 2 : c > 40 ? 4 : 8);
}

Plan plan_product(int R, int E, int N, int K, int group_size, bool summed) {
  const int experts = E == 0 ? 1 : E < R ? E : R;  // E = 0: one expert, R rows known to the host
  const double each = (double)R / experts;
  // (the first two kernels address an expert's packed words with 31 bits)
  if ((int64_t)N * K < ((int64_t)1 << 32)) {
    if (each <= (E == 0 ? 8 : 2)) return Plan{Plan::kFew, E == 0 && R > 4 ? 8 : 4, {}, {}};
    if (each <= (E == 0 ? 256 : 64)) return Plan{Plan::kStream, 0, plan_stream(R, experts, N, K), {}};
  }
  return Plan{Plan::kTiles, 0, {}, plan_tiles(R, experts, N, K, group_size, summed)};
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
