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

// One wave: 16 output columns (and their gate's partners) of a tile of 16
// rows, all of K.  v_mfma_f32_16x16x32_f16 with the weights as the A operand:
// lane (i, h) = (lane % 16, lane / 16) holds 8 channels of weight row i and
// of token row i, and the sums of token i with weight rows 4 h .. 4 h + 3.  The
// channels of a 128-channel step go to the lanes 32 at a time (one 128-bit
// load of packed words), the same way for both operands.
template <bool ZP, bool GATED>
__global__ __launch_bounds__(256) void product_kernel(PackedArgs w, ProductArgs p, int gshift, float* part) {
  constexpr int NB = GATED ? 2 : 1;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int li = lane & 15, lh = lane >> 4;
  const int width = GATED ? w.N >> 1 : w.N, G = w.K >> gshift;
  const int columns = (width + 63) / 64;  // blocks of 64 columns
  const int slot = blockIdx.x / columns, n0 = ((blockIdx.x - slot * columns) * 4 + wave) * 16;
  const RowTiles tiles(p.offsets, w.E, p.R, 16, 16);
  if (slot >= tiles.total) return;
  const RowTile t = tiles[slot];
  if (t.count <= 0 || n0 >= width) return;
  const DecodeConsts kc;
  int r = t.row0 + min(li, t.count - 1);
  if (p.rows) r = min(max(p.rows[r] / p.slots_per_row, 0), p.x_rows - 1);
  const _Float16* x = p.x + r * p.ldx;
  const size_t e = t.expert;
  const uint32_t* qw[NB];
  const uint16_t* sc[NB];
  const uint32_t* qz[NB];
  int zs[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int n = b * width + min(n0 + li, width - 1);
    qw[b] = w.qweight + (e * w.N + n) * (w.K >> 3);
    sc[b] = w.scales + e * w.N * G + scale_index(n, 0, G);
    qz[b] = ZP ? w.qzeros + e * (w.N >> 3) * G + zero_word_index(n, 0, G) : nullptr;
    zs[b] = 4 * (n & 7);
  }
  float4_t acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = float4_t{0.f, 0.f, 0.f, 0.f};
  for (int k = 32 * lh; k < ((w.K + 127) & ~127); k += 128) {
    const bool in = k < w.K;
    u32x4 xv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      xv[i] = in ? *reinterpret_cast<const u32x4*>(x + k + 8 * i) : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int g = min(k, w.K - 1) >> gshift;
      const u32x4 wv = in ? *reinterpret_cast<const u32x4*>(qw[b] + (k >> 3)) : u32x4{0, 0, 0, 0};
      const ZeroBias zb = zero_bias(ZP ? (qz[b][g] >> zs[b]) & 15u : 8u);
      const half2_t s2 = splat2(__builtin_bit_cast(_Float16, sc[b][(size_t)g * 8]));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(decode_word_scaled(wv[i], zb, kc, s2), as_half8(xv[i]), acc[b],
                                                        0, 0, 0);
    }
  }
  const int n = n0 + 4 * lh;
  if (li >= t.count || n >= width) return;
  const int64_t row = t.row0 + li;
  half4_t out;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float v = acc[0][j];
    if (p.bias) v += (float)p.bias[e * w.N + n + j];
    v = activate(v, p.activation);
    if constexpr (GATED) {
      float u = acc[NB - 1][j];
      if (p.bias) u += (float)p.bias[e * w.N + width + n + j];
      v *= u;
    }
    if (p.residual) v += (float)p.residual[row * p.ldr + n + j];
    if (part) part[row * width + n + j] = v;
    out[j] = (_Float16)v;
  }
  if (!part) *reinterpret_cast<half4_t*>(p.y + row * p.ldy + n) = out;
}

// part[row][n .. n + 3] summed over the K slices in order.
__device__ __forceinline__ float4_t slices_sum(const float* __restrict__ part, int splits, int64_t rows, int N,
                                               int64_t row, int n) {
  float4_t v = *reinterpret_cast<const float4_t*>(part + row * N + n);
  for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const float4_t*>(part + (s * rows + row) * N + n);
  return v;
}

// The epilogue of a product whose K was split: four columns per thread.
__global__ __launch_bounds__(256) void finish_kernel(const float* __restrict__ part, int splits, PackedArgs w,
                                                     ProductArgs p) {
  const int width = p.gated ? w.N >> 1 : w.N, quads = width >> 2;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / quads;
  const int n = (int)(i - row * quads) * 4;
  if (row >= p.R || (p.offsets && row >= min(p.offsets[w.E], p.R))) return;
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

// y[t] = sum over the slots j, in order, of weights[t][j] * part[positions[t][j]]
// + residual[t], four columns per thread.
__global__ __launch_bounds__(256) void combine_kernel(const float* __restrict__ part, int splits, CombineArgs c, int R,
                                                      int N) {
  const int quads = N >> 2;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)c.T * quads) return;
  const int64_t t = i / quads;
  const int n = (int)(i - t * quads) * 4;
  float4_t sum = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < c.top_k; ++j) {
    const int at = c.positions[t * c.top_k + j];
    if (at < 0 || at >= R) continue;
    sum += c.weights[t * c.top_k + j] * slices_sum(part, splits, R, N, at, n);
  }
  half4_t out;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (c.residual) sum[k] += (float)c.residual[t * c.ldr + n + k];
    out[k] = (_Float16)sum[k];
  }
  *reinterpret_cast<half4_t*>(c.y + t * c.ldy + n) = out;
}

hipError_t launch_rows(const PackedArgs& w, const ProductArgs& p, float* part, hipStream_t stream) {
  const int width = p.gated ? w.N / 2 : w.N, gs = log2_group(w.group_size);
  const dim3 grid((width + 63) / 64 * (p.offsets ? row_tiles(p.R, w.E, 16) : (p.R + 15) / 16));
  const auto kernel = w.qzeros ? (p.gated ? product_kernel<true, true> : product_kernel<true, false>)
                               : (p.gated ? product_kernel<false, true> : product_kernel<false, false>);
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, w, p, gs, part);
  return hipGetLastError();
}

// More than this many rows per expert on average: matrix-core tiles.
constexpr int kFewRows = 64;

struct Plan {
  bool tiles;
  TilePlan tile;
};

// Tile height and K split of the matrix-core tiles, from a time model: rounds of
// workgroups over the compute units, each a tile's steps (a 64-channel step of
// 256 rows 1.75 us, of 128 rows 1.0, of 64 rows 0.66: 0.29 + 0.18 per 32 rows)
// and ~6 us to begin and end it (256 weight rows, gated or not); with K split, the fp32 partials written and
// read at ~4 TB/s and one more launch.
TilePlan plan_tiles(int R, int experts, int N, int K) {
  const int steps = (K + 63) / 64, columns = (N + 255) / 256;
  constexpr double kUnits = 256;
  TilePlan best{256, 1, steps};
  double best_us = 1e300;
  for (int rows : {256, 128, 64}) {
    // ragged experts end in half a tile each on average
    const double tiles = experts == 1 ? (R + rows - 1) / rows : experts * ((double)R / experts / rows + 0.5);
    const double height = R / tiles / 32;
    const double step_us = 0.29 + 0.18 * (experts == 1 ? ceil(height) : height < 2 ? 2 : height);
    for (int s = 1; s <= 16 && s <= steps; ++s) {
      const int per = (steps + s - 1) / s, splits = (steps + per - 1) / per;
      const double rounds = ceil(tiles * columns * splits / kUnits);
      const double us = rounds * (per * step_us + 6.0) + (splits > 1 ? splits * (double)R * N * 8 / 4e6 + 3.0 : 0.0);
      if (us < best_us) best_us = us, best = TilePlan{rows, splits, per};
    }
  }
  return best;
}

Plan plan_product(int R, int E, int N, int K) {
  const int experts = E == 0 ? 1 : E < R ? E : R;  // E = 0: one expert, R rows known to the host
  if (R / experts <= kFewRows) return Plan{false, {0, 1, 0}};
  return Plan{true, plan_tiles(R, experts, N, K)};
}

size_t part_bytes(const Plan& plan, int R, int N) {
  return gemm_counter_bytes() + (size_t)(plan.tiles ? plan.tile.splits : 1) * R * N * 4;
}

float* part_of(void* workspace) {
  return reinterpret_cast<float*>(static_cast<char*>(workspace) + gemm_counter_bytes());
}

hipError_t launch_planned(const PackedArgs& w, const ProductArgs& p, const Plan& plan, float* part,
                          hipStream_t stream) {
  return plan.tiles ? launch_tiles(w, p, log2_group(w.group_size), plan.tile, part, stream)
                    : launch_rows(w, p, part, stream);
}

}  // namespace

size_t product_workspace_bytes(int R, int E, int N, int K, bool) {
  const Plan plan = plan_product(R, E, N, K);
  return plan.tiles && plan.tile.splits > 1 ? part_bytes(plan, R, N) : 0;
}

hipError_t launch_product(const PackedArgs& w, const ProductArgs& p, void* workspace, hipStream_t stream) {
  const Plan plan = plan_product(p.R, p.offsets ? w.E : 0, w.N, w.K);
  if (!plan.tiles || plan.tile.splits <= 1) return launch_planned(w, p, plan, nullptr, stream);
  float* part = part_of(workspace);
  const hipError_t e = launch_planned(w, p, plan, part, stream);
  if (e != hipSuccess) return e;
  const int64_t quads = (int64_t)p.R * ((p.gated ? w.N / 2 : w.N) / 4);
  hipLaunchKernelGGL(finish_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, stream, part, plan.tile.splits,
                     w, p);
  return hipGetLastError();
}

size_t combine_workspace_bytes(int T, int top_k, int E, int N, int K) {
  return part_bytes(plan_product(T * top_k, E, N, K), T * top_k, N);
}

hipError_t launch_combine(const PackedArgs& w, const ProductArgs& p, const CombineArgs& c, void* workspace,
                          hipStream_t stream) {
  const Plan plan = plan_product(p.R, w.E, w.N, w.K);
  float* part = part_of(workspace);
  const hipError_t e = launch_planned(w, p, plan, part, stream);
  if (e != hipSuccess) return e;
  const int64_t quads = (int64_t)c.T * (w.N / 4);
  hipLaunchKernelGGL(combine_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, stream, part,
                     plan.tiles ? plan.tile.splits : 1, c, p.R, w.N);
  return hipGetLastError();
}

}  // namespace awq
