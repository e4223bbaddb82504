// Shared by the fused layer (awq_linear_fused) and the expert products
// (awq_linear_experts, awq_combine_experts): how a workgroup finds the rows it
// multiplies, and what happens to a sum before it is stored.
#pragma once

#include "awq_device.hpp"
#include "awq_launch.hpp"

namespace awq {

typedef _Float16 half4_t __attribute__((ext_vector_type(4)));

// v = act(v) in fp32.  Each form passes NaN on; silu and the two gelus are
// written with one exponential (or erf) of the argument.
__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + __expf(-v)); }
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case 1: return v < 0.0f ? 0.0f : v;
    case 2: return v * sigmoid(v);
    case 3: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    // 0.5 v (1 + tanh u) = v sigmoid(2 u), u = sqrt(2 / pi) (v + 0.044715 v^3)
    case 4: return v * sigmoid(1.5957691216057308f * (v + 0.044715f * v * v * v));
    default: return v;
  }
}

// The rows of one workgroup: `count` consecutive rows from `row0`, all of
// expert `expert` (count 0: the workgroup has nothing to do).
struct RowTile {
  int expert, row0, count;
};

// Tile `slot` of the rows sorted by expert, cut into tiles of at most `tile`
// rows of one expert each: expert e holds the rows offsets[e] ..
// offsets[e + 1] - 1.  The counts live on the device only, so the host launches
// row_tiles(R, E, tile) tiles and each wave finds its own here, 64 experts at a
// time: lane l counts expert l's tiles, a prefix sum over the lanes places them,
// and the first lane whose sum passes `slot` is the expert.  Offsets are
// clamped into [0, R], so no wrong value leads outside the buffers.
__device__ __forceinline__ RowTile find_row_tile(const int* __restrict__ offsets, int E, int R, int tile, int slot) {
  if (offsets == nullptr) return RowTile{0, slot * tile, min(tile, R - slot * tile)};
  const int lane = __lane_id();
  int seen = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, n = 0;
    if (e < E) {
      lo = min(max(offsets[e], 0), R);
      n = max(min(offsets[e + 1], R) - lo, 0);
    }
    int sum = (n + tile - 1) / tile;  // inclusive prefix sum over the lanes
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    const unsigned long long past = __ballot(seen + sum > slot);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      const int elo = __builtin_amdgcn_readlane(lo, l), en = __builtin_amdgcn_readlane(n, l);
      const int before = seen + __builtin_amdgcn_readlane(sum, l) - (en + tile - 1) / tile;
      const int first = (slot - before) * tile;
      return RowTile{e0 + l, elo + first, min(tile, en - first)};
    }
    seen += __builtin_amdgcn_readlane(sum, 63);
  }
  return RowTile{0, 0, 0};
}

// Most tiles that R rows of E experts can take: every expert but the last
// has one row, or all rows fill tiles and every expert has one ragged tile.
__host__ __device__ inline int row_tiles(int R, int E, int tile) {
  return R <= E ? R : E + (R - E) / tile;
}

}  // namespace awq
