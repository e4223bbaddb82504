// Shared by the kernels on a paged cache of keys and values: which sequence,
// place, page and slot a row belongs to.
//
// The numbers live on the device only, and wrong ones must not lead outside the
// buffers: rows are clamped into [0, T], lengths into [0, width * S], page
// numbers into [0, pages) for reading (wrong results), and nothing is written to a
// page whose number is out of range.
#pragma once

#include "awq_epilogue.hpp"
#include "awq_launch_cache.hpp"

namespace awq {

// The rows of one sequence and the place of the first of them.
struct Sequence {
  int index, row0, rows, length;
  __device__ __forceinline__ int place0() const { return length - rows; }  // below 0: rows without a place
};

__device__ __forceinline__ Sequence sequence_at(const SeqArgs& s, int shift, int b) {
  Sequence q{b, 0, 0, 0};
  if (b < s.B) {
    q.row0 = min(max(s.offsets[b], 0), s.T);
    q.rows = max(min(s.offsets[b + 1], s.T) - q.row0, 0);
    q.length = (int)min((int64_t)max(s.lengths[b], 0), (int64_t)s.width << shift);
  }
  return q;
}

__device__ __forceinline__ Sequence pick(const Sequence& q, int lane) {
  return Sequence{__builtin_amdgcn_readlane(q.index, lane), __builtin_amdgcn_readlane(q.row0, lane),
                  __builtin_amdgcn_readlane(q.rows, lane), __builtin_amdgcn_readlane(q.length, lane)};
}

// The sequence that row t belongs to (rows 0: none does).  One wave, 64
// sequences at a time.
__device__ __forceinline__ Sequence sequence_of(const SeqArgs& s, int shift, int t) {
  for (int b0 = 0; b0 < s.B; b0 += 64) {
    const Sequence q = sequence_at(s, shift, b0 + __lane_id());
    const unsigned long long owner = __ballot(t >= q.row0 && t < q.row0 + q.rows);
    if (owner != 0) return pick(q, __builtin_ctzll(owner));
  }
  return Sequence{0, 0, 0, 0};
}

__device__ __forceinline__ int page_number(const CacheArgs& c, int page) { return min(max(page, 0), c.pages - 1); }

}  // namespace awq
