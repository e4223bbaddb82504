// Attention of many rows (prompts, and the shared keys of a batch): workgroups of
// 128 rows, four waves of 32, that share each block of keys and values.
//
// Mathematics: awq_attend_block.hpp's.  A row is a token and a query head of one key
// head, so the query heads of a group and, for the shared keys, the sequences of the
// batch are rows of one product: the shared keys are read once per 128 rows, not
// once per sequence.
//
// Bound: the matrix cores (4 D operations per row and key) beside the
// exponentials: 13 questions after 16384 shared tokens 496-542 us back to back with their
// join, 0.92-1.0 PFLOP/s by the part, with two workgroups per unit at the power limit
// (549-588 without it in a trace, at lower clocks); a wave that has its SIMD to
// itself takes 0.8 us per block (a prompt of 2000, whose last tiles see 64 of them: 54
// us).  A block of keys and values goes straight to LDS while the one before it is
// multiplied, with one barrier per block.  Where the row tiles are
// too few for the chip, the keys are split as well and the parts joined by a second
// launch.
#pragma once

#include "awq_attend.hpp"

namespace awq {

template <int D>
struct TileRing {
  static constexpr int BLOCKS = 4, BYTES = 2 * BLOCKS * 32 * Tile<D>::ROW;
};

// All rows of the batch as one sequence that ends with the shared keys, with the table of the first that has rows (those
// before it need not have any pages); `within`: one of those with rows among tokens t0 to t1 has new tokens among the
// shared keys, which see only those up to their own places.
struct SharedRows {
  Sequence all;
  bool within;
};
__device__ __forceinline__ Sequence all_tokens(const SeqArgs& s, int shared_keys) {
  const int from = min(max(s.offsets[0], 0), s.T);
  return Sequence{0, from, max(min(s.offsets[s.B], s.T) - from, 0), shared_keys};
}
__device__ __forceinline__ SharedRows shared_rows(const SeqArgs& s, int shift, Sequence all, int t0, int t1) {
  SharedRows r{all, false};
  bool found = false;
  for (int b0 = 0; b0 < s.B; b0 += 64) {
    const Sequence q = sequence_at(s, shift, b0 + __lane_id());
    const unsigned long long some = __ballot(q.rows > 0);
    if (!found && some != 0) {
      r.all.index = b0 + __builtin_ctzll(some);
      found = true;
    }
    r.within = r.within || __any(q.rows > 0 && q.row0 <= t1 && q.row0 + q.rows > t0 && q.place0() < all.length);
  }
  return r;
}
// Where the lane's token t is among the shared keys (the last of them, or its own place if that is before it), of tokens
// t0 to t1, and the least such place.
__device__ __forceinline__ int shared_place(const SeqArgs& s, int shift, int last, int t, int t0, int t1, int& least) {
  int place = last;
  least = last;
  for (int b0 = 0; b0 < s.B; b0 += 64) {
    const Sequence q = sequence_at(s, shift, b0 + __lane_id());
    unsigned long long here = __ballot(q.rows > 0 && q.row0 <= t1 && q.row0 + q.rows > t0 && q.place0() < last);
    while (here != 0) {
      const Sequence of = pick(q, __builtin_ctzll(here));
      here &= here - 1;
      if (t >= of.row0 && t < of.row0 + of.rows) place = min(place, of.place0() + t - of.row0);
      least = min(least, of.place0() + max(t0 - of.row0, 0));
    }
  }
  return place;
}

// Workgroup number `index` of 256 threads; a ring of TileRing<D>::BYTES and two words.
template <int D>
__device__ __forceinline__ void attend_tile(const AttendArgs& a, const CacheArgs& c, const SeqArgs& s, const TileArgs& x,
                                            const Partials& p, int index, lds_char* ring, uint32_t* strange) {
  using T = Tile<D>;
  // Blocks of 32 keys in a ring: a block's scores are made beside the weights of the one before (matrix and vector
  // instructions of one wave), with two blocks on their way.
  constexpr int RING = TileRing<D>::BLOCKS, LOADS = T::LOADS, SLOT = 32 * T::ROW;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), group = x.group;
  const float scale = a.scale * kLog2E;

  // the tile: key heads next to each other (one XCD keeps meeting the same); the last rows, which have the most keys,
  // first, and where there are at most two workgroups per compute unit the second ones the other way around, so that
  // each unit gets one with many keys and one with few; numbers that no rows have (the host knows a bound only) all at
  // one end, so that the XCDs, which take workgroups in turn, get equally many that have some
  const int head = index % c.heads;
  int nth = index / c.heads;
  const bool shared = nth < x.shared_tiles * x.shared_splits;
  int split, splits, slice, key0, keys;
  Rows rows;  // of the workgroup, then of the wave
  Sequence seq;
  int token0 = 0, token1 = 0;  // of the shared keys: the workgroup's first and last
  bool within = false;
  if (shared) {
    split = nth / x.shared_tiles;
    splits = x.shared_splits;
    slice = x.shared_slice + split;
    seq = all_tokens(s, a.shared);
    rows = Rows{kTile * (nth - split * x.shared_tiles), seq.rows * group, seq.row0, 0};
    if (rows.first >= rows.total) return;
    token0 = seq.row0 + rows.first / group;
    token1 = seq.row0 + (min(rows.first + kTile, rows.total) - 1) / group;
    const SharedRows r = shared_rows(s, c.shift, seq, token0, token1);
    seq = r.all;
    within = r.within;
    key0 = 0;
    keys = a.shared;
  } else {
    nth -= x.shared_tiles * x.shared_splits;
    splits = x.own_splits;
    split = nth % splits;
    slice = x.own_slice < 0 ? -1 : x.own_slice + split;
    const int turn = nth / splits, wanted = turn < x.descending ? x.own_tiles - 1 - turn : turn - x.descending;
    int seen = 0;
    bool found = false;
    for (int b0 = 0; b0 < s.B; b0 += 64) {
      const Sequence q = sequence_at(s, c.shift, b0 + lane);
      const int tiles = (q.rows * group + kTile - 1) / kTile, sum = seen + prefix_sum(tiles);
      const unsigned long long owner = __ballot(sum > wanted && sum - tiles <= wanted);
      if (owner != 0) {
        const int l = __builtin_ctzll(owner);
        seq = pick(q, l);
        rows = Rows{kTile * (wanted - __builtin_amdgcn_readlane(sum - tiles, l)), seq.rows * group, seq.row0, seq.place0()};
        found = true;
        break;
      }
      seen = __builtin_amdgcn_readlane(sum, 63);
    }
    if (!found) return;
    key0 = a.shared;
    keys = rows.place0 + (min(rows.first + kTile, rows.total) - 1) / group + 1 - key0;
  }
  const int blocks = keys > 0 ? (keys + 31) / 32 : 0;
  const int from = (int)((long long)blocks * split / splits), to = (int)((long long)blocks * (split + 1) / splits);

  // least and greatest place of the workgroup's rows
  int tile_least = shared ? a.shared - 1 : rows.place0 + rows.first / group;
  const int tile_most = key0 + keys - 1;
  if (threadIdx.x < 2) strange[threadIdx.x] = 0;
  rows.first += 32 * wave;
  const bool live = rows.first < rows.total;
  const int mine = min(rows.first + (lane & 31), rows.total - 1) / group;
  int place = shared ? a.shared - 1 : rows.place0 + mine;
  int least = shared ? a.shared - 1 : rows.place0 + min(rows.first, rows.total - 1) / group;
  if (within) {
    place = shared_place(s, c.shift, a.shared - 1, seq.row0 + mine, token0, token1, tile_least);
    least = tile_least;
  }

  Queries<D, 32> q;
  read_queries(q, a, rows, group, head);
  Gathered<D, 32> g;
  g.clear();

  // this wave's loads of a block: of keys or of values, one group of 16 of them
  const int sixteen = wave & 1, of_values = wave >> 1;
  uint32_t lane_from[LOADS];
  {
    const Sources<D> sources(lane);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) lane_from[i] = of_values ? sources.value(i) : sources.key(i);
  }
  const Addresses<D, 32> places((uint32_t)(uintptr_t)ring, lane);
  Entries pages{s.tables + (int64_t)seq.index * s.width, nullptr, 0, s.width, head, 0, 0, 0, 0};
  auto source_of = [&](int block) __attribute__((always_inline)) {
    const int key = key0 + 32 * block;
    if (block == from || ((key + 16) >> c.shift) - pages.first >= 64) pages.read(c, key >> c.shift);
    return reinterpret_cast<const char*>((of_values ? c.v : c.k) + keys16(pages, c, key + 16 * sixteen).at * D);
  };
  lds_char* const own = ring + of_values * SLOT + 16 * sixteen * T::ROW;
  auto meet = [&]() __attribute__((always_inline)) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // past the least place of the workgroup's rows some values are not to be seen by some row
  auto hide = [&](int block, int slot) __attribute__((always_inline)) {
    const int key = key0 + 32 * block;
    if (key + 31 <= tile_least) return 0u;  // (the same for the whole workgroup)
    const uint32_t met = (uint32_t)hide_strange<D, 32>(ring + (2 * slot + 1) * SLOT, threadIdx.x, 256,
                                                       [&](int h, int& behind, int& upto) {
                                                         behind = tile_least - key - 16 * h;
                                                         upto = tile_most - key - 16 * h;
                                                       });
    if (met) atomicOr(&strange[block & 1], met);
    if (threadIdx.x == 0) strange[(block + 1) & 1] = 0;
    meet();
    return (uint32_t)__builtin_amdgcn_readfirstlane(strange[block & 1]);
  };
  auto seen_of = [&](int block) __attribute__((always_inline)) {
    const int key = key0 + 32 * block;
    return Seen{place - key, place - key - 16, least - key >= 31};
  };
  auto finish = [&](int block, uint32_t odd, const Weights<32>& p, const Seen& seen) __attribute__((always_inline)) {
    if (__builtin_expect(odd != 0, 0))
      gather_strange<D, 32>(odd, p, seen, [&](int k) {
        const int key = key0 + 32 * block + k;
        const int64_t number = page_number(c, pages.table[key >> c.shift]);
        return c.v + (((number * c.heads + head) << c.shift) + (key & ((1 << c.shift) - 1))) * D;
      }, g);
  };
  Scores<32> s_now{};
  float m_now = 0.0f;
  if (from < to) {
#pragma unroll
    for (int i = 0; i < RING - 1; ++i) {
      const char* base = source_of(min(from + i, to - 1));
#pragma unroll
      for (int n = 0; n < LOADS; ++n) load_to_lds<1>(base, {lane_from[n]}, own + 2 * SLOT * i + 1024 * n);
    }
    wait_loads<(RING - 2) * LOADS>();
    meet();
    Fragments f = first_keys<D, 32, 0>(places);
    s_now = scores_of<D, 32, 0>(places, q, f, [](auto) __attribute__((always_inline)) {});
    m_now = greatest(s_now);
  }
  // One block: its scores are there, the next block's are made; the one after that may still be on its way, and the
  // fourth takes the place of the last (past the end, the last block again: its scores count nothing).
  auto step = [&](int block, auto slot, auto plain) __attribute__((always_inline)) {
    asm volatile("" : "+v"(s_now.s));  // (keeps the scores of both loops below in the same two sets of registers)
    constexpr int HERE = decltype(slot)::value, NEXT = (HERE + 1) % RING;
    wait_loads<(RING - 3) * LOADS>();
    meet();
    Fragments f = first_keys<D, 32, 2 * NEXT * SLOT>(places);
    const char* base = source_of(min(block + RING - 1, to - 1));
    uint32_t odd = 0;
    Seen seen{0, 0, true};
    if constexpr (!decltype(plain)::value) {
      odd = hide(block, HERE);
      seen = seen_of(block);
    }
    const Weights<32> p = attend_next<D, 32, 2 * NEXT * SLOT, (2 * HERE + 1) * SLOT>(
        places, q, f, scale, seen, s_now, m_now, g, [&](auto n) __attribute__((always_inline)) {
          constexpr int i = decltype(n)::value;
          static_assert(Products<D, 32>::VALUES == 2 * LOADS, "a load for every other of them");
          load_to_lds<1>(base, {lane_from[i]}, own + 2 * SLOT * ((HERE + RING - 1) % RING) + 1024 * i);
        });
    if constexpr (!decltype(plain)::value) finish(block, odd, p, seen);
  };
  // Blocks that all rows see whole, four at a time, without a thought for what some must not see (with both in one loop
  // the scores are copied for every block).
  const int whole = max(tile_least - key0 + 1, 0) / 32;
  int block = from;
  for (; block + RING <= min(whole, to); block += RING)
    each<0, RING, 1>([&](auto slot) __attribute__((always_inline)) {
      step(block + decltype(slot)::value, slot, std::true_type{});
    });
  for (; block < to; block += RING)
    each<0, RING, 1>([&](auto slot) __attribute__((always_inline)) {
      constexpr int i = decltype(slot)::value;
      if (block + i < to) step(block + i, slot, std::false_type{});
    });
  wait_loads<0>();  // (those past the end)
  if (live) write_rows(g, a, p, rows, group, head, slice, nullptr, nullptr);
}

}  // namespace awq
