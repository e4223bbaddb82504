// Shared by the fused layer (awq_linear_fused) and the expert products
// (awq_linear_experts, awq_combine_experts): how a workgroup finds the rows it
// multiplies, and what happens to a sum before it is stored.
#pragma once

#include "awq_device.hpp"
#include "awq_launch.hpp"
#include "awq_launch_fused.hpp"

namespace awq {

typedef _Float16 half4_t __attribute__((ext_vector_type(4)));

// v = act(v) in fp32.  Each form passes NaN on; silu and the two gelus are
// written with one exponential (or erfc) of the argument, and no form adds numbers
// that cancel: the small values below zero keep their relative accuracy, which a
// gate's other factor carries back into fp16's range.
__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + __expf(-v)); }
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case 1: return v < 0.0f ? 0.0f : v;
    case 2: return v * sigmoid(v);
    case 3: return 0.5f * v * erfcf(v * -0.70710678118654752f);
    // 0.5 v (1 + tanh u) = v sigmoid(2 u), u = sqrt(2 / pi) (v + 0.044715 v^3)
    case 4: return v * sigmoid(1.5957691216057308f * (v + 0.044715f * v * v * v));
    default: return v;
  }
}

template <int ACT>
__device__ __forceinline__ void activate8_as(float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = activate(v[k], ACT);
}
__device__ __forceinline__ void activate8(float (&v)[8], int act) {
  switch (act) {
    case 1: return activate8_as<1>(v);
    case 2: return activate8_as<2>(v);
    case 3: return activate8_as<3>(v);
    case 4: return activate8_as<4>(v);
    default: return;
  }
}

// Eight consecutive outputs n .. n + 7 of row r: bias, activation, gate and
// residual on the fp32 sums v (and u, the gate's partners), one rounding.
template <bool GATED>
__device__ __forceinline__ void finish8(float (&v)[8], const float (&u)[8], const ProductArgs& p, size_t wrow, int width,
                                        int64_t r, int n, int act) {
  half8_t b, ub, res, out;
  if (p.bias) {
    b = *reinterpret_cast<const half8_t*>(p.bias + wrow + n);
    if constexpr (GATED) ub = *reinterpret_cast<const half8_t*>(p.bias + wrow + width + n);
  }
  if (p.residual) res = *reinterpret_cast<const half8_t*>(p.residual + r * p.ldr + n);
  if (p.bias)
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += (float)b[k];
  activate8(v, act);
  if constexpr (GATED) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= p.bias ? u[k] + (float)ub[k] : u[k];
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) out[k] = (_Float16)(p.residual ? v[k] + (float)res[k] : v[k]);
  *reinterpret_cast<half8_t*>(p.y + r * p.ldy + n) = out;
}

// The rows of one workgroup: `count` consecutive rows from `row0`, all of
// expert `expert` (count 0: the workgroup has nothing to do).
struct RowTile {
  int expert, row0, count;
};

// Sum of v over this lane and the lanes below it, in registers (DPP shifts
// within 16 lanes, then the last lane of each 16 and 32 to those above).
__device__ __forceinline__ int prefix_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31
  return v;
}

// 64 experts' row ranges and tiles, one expert per lane.
struct ExpertLanes {
  int lo, n, tiles, sum;  // first row, rows, tiles, one past the number of the last of them
};
__device__ __forceinline__ ExpertLanes expert_lanes(const int* __restrict__ offsets, int E, int R, int tile, int e0) {
  const int e = e0 + __lane_id();
  ExpertLanes x{0, 0, 0, 0};
  if (e < E) {
    x.lo = min(max(offsets[e], 0), R);
    x.n = max(min(offsets[e + 1], R) - x.lo, 0);
  }
  x.tiles = (x.n + tile - 1) / tile;
  x.sum = prefix_sum(x.tiles);
  return x;
}

// The rows sorted by expert (expert e: offsets[e] .. offsets[e + 1] - 1), cut into
// tiles of at most `tile` rows of one expert each, an expert's units of `unit`
// rows shared evenly among its tiles (`tile` a multiple of `unit`).  The counts live on
// the device only, so the host launches for row_tiles(R, E, tile) tiles and
// each wave finds its own here, 64 experts at a time: lane l counts expert l's
// tiles, a prefix sum over the lanes numbers them, and the lane whose numbers
// hold the wanted tile is the expert.  Offsets are clamped into [0, R], so no
// wrong value leads outside the buffers.  With `offsets` NULL one expert holds
// all R rows.
struct RowTiles {
  const int* offsets;
  int E, R, tile, unit, total;
  ExpertLanes first;  // the first 64 experts

  __device__ __forceinline__ RowTiles(const int* o, int experts, int rows, int t, int u)
      : offsets(o), E(experts), R(rows), tile(t), unit(u), first{0, 0, 0, 0} {
    if (offsets == nullptr) {
      total = (R + tile - 1) / tile;
      return;
    }
    first = expert_lanes(offsets, E, R, tile, 0);
    total = __builtin_amdgcn_readlane(first.sum, 63);
    for (int e0 = 64; e0 < E; e0 += 64)
      total += __builtin_amdgcn_readlane(expert_lanes(offsets, E, R, tile, e0).sum, 63);
  }

  __device__ __forceinline__ RowTile cut(int expert, int lo, int n, int tiles, int nth) const {
    if (tiles == 1) return RowTile{expert, lo, n};
    const int units = (n + unit - 1) / unit, each = units / tiles, more = units - each * tiles;
    const int from = unit * (nth * each + min(nth, more));
    return RowTile{expert, lo + from, min(unit * (each + (nth < more)), n - from)};
  }

  // Numbers the tiles of up to 64 experts by height: the experts with the
  // tallest tiles first.
  __device__ __forceinline__ void tallest_first() {
    if (offsets == nullptr || E > 64) return;
    const int units = (first.n + unit - 1) / unit, height = first.tiles ? (units + first.tiles - 1) / first.tiles : 0;
    int before = 0;
    for (int e = 0; e < E; ++e) {
      const int h = __builtin_amdgcn_readlane(height, e), tiles = __builtin_amdgcn_readlane(first.tiles, e);
      before += h > height || (h == height && e < (int)__lane_id()) ? tiles : 0;
    }
    first.sum = before + first.tiles;
  }

  // 0 <= slot < total
  __device__ __forceinline__ RowTile operator[](int slot) const {
    if (offsets == nullptr) return cut(0, 0, R, total, slot);
    int seen = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const ExpertLanes x = e0 == 0 ? first : expert_lanes(offsets, E, R, tile, e0);
      const unsigned long long owner = __ballot(seen + x.sum > slot && seen + x.sum - x.tiles <= slot);
      if (owner != 0) {
        const int l = __builtin_ctzll(owner);
        const int tiles = __builtin_amdgcn_readlane(x.tiles, l);
        return cut(e0 + l, __builtin_amdgcn_readlane(x.lo, l), __builtin_amdgcn_readlane(x.n, l), tiles,
                   slot - (seen + __builtin_amdgcn_readlane(x.sum, l) - tiles));
      }
      seen += __builtin_amdgcn_readlane(x.sum, 63);
    }
    return RowTile{0, 0, 0};
  }
};

// Most tiles that R rows of E experts can take: every expert but the last
// has one row, or all rows fill tiles and every expert has one ragged tile.
__host__ __device__ inline int row_tiles(int R, int E, int tile) {
  return R <= E ? R : E + (R - E) / tile;
}

}  // namespace awq
