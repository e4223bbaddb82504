// How the attention kernels share a batch's work, and where they leave what is
// to be joined.
#pragma once

#include "awq_attend_block.hpp"

namespace awq {

constexpr int kUnits = 256;  // compute units
// Waves on their own of a unit, each with a ring of two blocks.  (With five a unit's LDS is full, and HBM serves their
// many streams less well: 1 token of 8191 40.5 us, with two 32.4; 48 tokens 103, 96, with four 93.4; 32 tokens on chosen
// pages 102, 92; 1 token of 30000 46, 36.  Rings of three or four blocks: the same or slower.  With one, two, four at
// the other head sizes, 1 token of 8191 / 48 tokens: of 64 25.9, 18.4, 18.8 / 86, 56, 53; of 96 29.9, 24.3, 25.5 / 99, 76, 73; of
// 256, where a unit has room for two, 32.9, 35.1, 43.0 / 184, 174, 178.)
constexpr int kWavesOfUnit = 2, kWaves = kUnits * kWavesOfUnit;
constexpr int kLeastUnits = 2;  // key blocks that a wave takes at least

// Rows of 16 or 32 and keys of 32 of one wave (few), rows of 128 and splits of the keys (many, and all shared keys).
struct AttendPlan {
  bool own_few;  // a sequence's own keys: with the waves, or with the workgroups
  bool shared;   // there are shared keys
  int rows;      // of a wave: 16 or 32
  int own_splits, shared_splits;  // of the workgroups
  bool both() const { return own_few && shared; }  // in one launch
  int own_slices() const { return own_few ? shared : shared || own_splits > 1 ? own_splits : 0; }
  int slices() const { return own_slices() + (shared ? shared_splits : 0); }
};

// Partial results: for each row's query head (numbered t * q_heads + head) and slice the maximum (of the scores as they
// are, which differ exactly), the sum and the values' sums: slice 0 (to own_splits - 1) the own keys, the rest the shared
// ones; and two of those of 32 rows per wave (or of its 16), for a piece that starts within a segment and one that ends within one.
struct Partials {
  float2* stat;    // [slices][rows]
  float* sums;     // [slices][rows][dim]
  float2* wave_stat;  // [waves][2][32]
  float* wave_sums;   // [waves][2][32][dim]
  int64_t rows;
};

inline Partials partials(const AttendPlan& p, int64_t rows, int dim, void* workspace) {
  Partials x;
  const int64_t waves = p.own_few ? 64 * kWaves : 0;
  x.rows = rows;
  x.sums = static_cast<float*>(workspace);
  x.wave_sums = x.sums + p.slices() * rows * dim;
  x.stat = reinterpret_cast<float2*>(x.wave_sums + waves * dim);
  x.wave_stat = x.stat + p.slices() * rows;
  return x;
}
inline size_t partial_bytes(const AttendPlan& p, int64_t rows, int dim) {
  const int64_t all = p.slices() * rows + (p.own_few ? 64 * kWaves : 0);
  return ((size_t)all * (dim * 4 + 8) + 15) & ~(size_t)15;
}

hipError_t launch_attend_waves(const AttendArgs& a, const CacheArgs& c, const SeqArgs& s, const AttendPlan& plan,
                               const Partials& p, hipStream_t stream);
hipError_t launch_attend_tiles(const AttendArgs& a, const CacheArgs& c, const SeqArgs& s, const AttendPlan& plan,
                               const Partials& p, hipStream_t stream);

// How a plan's row tiles (kTile rows each) are numbered: `shared_tiles` workgroup rows of the shared keys first, then the
// sequences' own.
constexpr int kTile = 128;
struct TileArgs {
  int group, shared_tiles, shared_splits, own_tiles, own_splits, own_slice, shared_slice;
  int descending;  // of the own tiles (per key head), those that come first, from the last rows up
};
inline TileArgs tile_args(const AttendPlan& plan, int T, int B, int q_heads, int kv_heads, int dim) {
  const int group = q_heads / kv_heads;
  const int64_t rows = (int64_t)T * group, most = rows / kTile + B;  // (a ragged tile per sequence at most)
  TileArgs x{group, 0, 1, 0, 1, plan.own_slices() > 0 ? 0 : -1, plan.own_slices(), 0};
  if (plan.shared) {
    x.shared_tiles = (int)((rows + kTile - 1) / kTile);
    x.shared_splits = plan.shared_splits;
  }
  if (!plan.own_few) {
    x.own_tiles = (int)(most < rows ? most : rows);
    x.own_splits = plan.own_splits;
    const int first = (kUnits + kv_heads - 1) / kv_heads;
    const bool twice = x.shared_tiles == 0 && x.own_splits == 1 && x.own_tiles > first && x.own_tiles <= 2 * first;
    x.descending = twice && dim < 256 ? first : x.own_tiles;
  }
  return x;
}
inline int64_t tile_workgroups(const TileArgs& x, int kv_heads) {
  return ((int64_t)x.shared_tiles * x.shared_splits + (int64_t)x.own_tiles * x.own_splits) * kv_heads;
}

// The units of work of the waves (16 or 32 rows, a key head, 32 keys), in order: sequence after sequence; within one, rows,
// then key heads, then keys.  Every row has at least one.  Wave w takes the units w * each .. w * each + each - 1.  (The
// host makes sure that their number stays below kMostUnits.)
struct Units {
  int total, each;
};
struct UnitArgs {
  int group, heads, shift, shared_keys;
  int rows;  // of a unit: 16 or 32
};
inline UnitArgs unit_args(const AttendArgs& a, const CacheArgs& c, const AttendPlan& plan) {
  return UnitArgs{a.q_heads / c.heads, c.heads, c.shift, a.shared, plan.rows};
}
__device__ __forceinline__ int key_blocks(const UnitArgs& u, int length) { return max((length - u.shared_keys + 31) >> 5, 1); }
__device__ __forceinline__ int row_blocks(const UnitArgs& u, int rows) { return (rows * u.group + u.rows - 1) / u.rows; }
__device__ __forceinline__ int units_of(const UnitArgs& u, const Sequence& q) {
  return q.rows ? row_blocks(u, q.rows) * u.heads * key_blocks(u, q.length) : 0;
}
__device__ __forceinline__ Units share_units(int total) {
  return Units{total, max((total + kWaves - 1) / kWaves, kLeastUnits)};
}
__device__ __forceinline__ Units count_units(const SeqArgs& s, const UnitArgs& u) {
  int total = 0;
  for (int b0 = 0; b0 < s.B; b0 += 64)
    total += __builtin_amdgcn_readlane(prefix_sum(units_of(u, sequence_at(s, u.shift, b0 + __lane_id()))), 63);
  return share_units(total);
}
// For a list of pages per token: units of a token.
__device__ __forceinline__ int list_blocks(const UnitArgs& u, int count) { return ((count << u.shift) + 31) >> 5; }

constexpr int64_t kMostUnits = 1 << 30;

constexpr int kNowhere = 1 << 30;  // a place behind every row's (subtracting it stays in 32 bits)

// Rows, numbered token after token, the key head's query heads within one: `first` is the number of the first,
// `total` how many the sequence has; `place0` and `row0` are of its first token.
struct Rows {
  int first, total, row0, place0;
};

// The pages of a segment's keys, 64 entries of its table or list at a time, one per lane: where the key head's part of
// the page begins, and the place of its first token.
struct Entries {
  const int* table;  // the sequence's
  const int* list;   // or NULL: every page of the table
  int count, width;  // of the list, of the table
  int head;
  int first;              // entry of lane 0
  uint32_t at_lo, at_hi;  // row of the cache
  int place;

  __device__ __forceinline__ void read(const CacheArgs& c, int from) {
    first = from;
    const int e = from + (int)__lane_id();
    int page = list ? (e < count ? list[e] : -1) : e;
    if (page < 0 || page >= width) page = -1;
    const uint64_t at = ((int64_t)page_number(c, page >= 0 ? table[page] : 0) * c.heads + head) << c.shift;
    at_lo = (uint32_t)at;
    at_hi = (uint32_t)(at >> 32);
    place = page < 0 ? kNowhere : page << c.shift;
  }
};

// Where 16 keys are, and the place of the first of them in the sequence.
struct Keys16 {
  int64_t at;  // row of the cache
  int place;
};
__device__ __forceinline__ Keys16 keys16(const Entries& e, const CacheArgs& c, int key) {
  const int lane = (key >> c.shift) - e.first, slot = key & ((1 << c.shift) - 1);
  const uint32_t lo = __builtin_amdgcn_readlane(e.at_lo, lane), hi = __builtin_amdgcn_readlane(e.at_hi, lane);
  return Keys16{(int64_t)((uint64_t)hi << 32 | (lo + slot)), __builtin_amdgcn_readlane(e.place, lane) + slot};
}

// The queries of a wave's R rows.
template <int D, int R>
__device__ __forceinline__ void read_queries(Queries<D, R>& q, const AttendArgs& a, const Rows& r, int group, int head) {
  const int lane = __lane_id(), row = r.first + (lane & (R - 1)), token = row / group;
  const bool live = row < r.total;
  const _Float16* from = a.q + (live ? (r.row0 + token) * a.ldq + (int64_t)(head * group + row - token * group) * D : 0) +
                         8 * (lane / R);
#pragma unroll
  for (int j = 0; j < Queries<D, R>::PARTS; ++j) {
    const half8_t v = *reinterpret_cast<const half8_t*>(from + 512 / R * j);
    q.part[j] = live ? v : half8_t((_Float16)0.0f);
  }
}

constexpr float kNoPlace = -1.0f;  // a sum that no row can have

// Results of a wave's R rows: to y (`slice` below 0), or unfinished to a slice of the rows, or to `wave_stat` and
// `wave_sums` of R rows.
template <int D, int R>
__device__ __forceinline__ void write_rows(const Gathered<D, R>& g, const AttendArgs& a, const Partials& p,
                                           const Rows& r, int group, int head, int slice, float2* wave_stat,
                                           float* wave_sums) {
  const int lane = __lane_id(), row = r.first + (lane & (R - 1)), token = row / group, h = lane / R;
  if (row >= r.total) return;
  const float sum = row_sum<R>(g.sum);
  const int64_t t = r.row0 + token;
  const int at = head * group + row - token * group;
  if (slice < 0 && !wave_stat) {
    const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
    _Float16* y = a.y + t * a.ldy + (int64_t)at * D + 4 * h;
#pragma unroll
    for (int n = 0; n < Gathered<D, R>::QUADS; ++n) {
      half4_t v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (_Float16)(sum == 0.0f ? 0.0f : g.get(n, i) * by);
      *reinterpret_cast<half4_t*>(y + 256 / R * n) = v;
    }
    return;
  }
  const int64_t to = wave_stat ? lane & (R - 1) : (int64_t)slice * p.rows + t * a.q_heads + at;
  // (a row without a place is marked: shared keys, which it does not have, must not count for it)
  if (h == 0)
    (wave_stat ? wave_stat : p.stat)[to] = r.place0 + token < 0 ? float2{0.0f, kNoPlace} : float2{g.top, sum};
  float* sums = (wave_stat ? wave_sums : p.sums) + to * D + 4 * h;
#pragma unroll
  for (int n = 0; n < Gathered<D, R>::QUADS; ++n) {
    float4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = g.get(n, i);
    *reinterpret_cast<float4_t*>(sums + 256 / R * n) = v;
  }
}

}  // namespace awq
