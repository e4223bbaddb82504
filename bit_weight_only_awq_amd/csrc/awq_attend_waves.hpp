// Attention of few rows per sequence (decoding): each wave on its own, 16 or 32 rows
// of queries against an equal share of all keys.
//
// Mathematics: awq_attend_block.hpp's.  A unit of work is 32 keys for up to R rows
// (tokens times query heads of one key head); all units of the batch, whatever the
// lengths, are one list, and each of kWaves waves takes an equal run of it, so
// ragged batches and single long sequences fill the chip alike.  A wave that
// takes a whole segment (rows, key head) writes its result; the pieces of the
// others are joined by a second launch.
//
// Bound: HBM, each key and value once (1 token of 8191, 134 MB: 24.5 us, 5.5 TB/s; 48
// tokens of up to 4000, 451 MB: 90 us, 5.0; 32 tokens on 64 chosen pages, 268 MB: 53
// us, 5.1).  Keys and values go straight to LDS
// (16 bytes per lane, whole rows), one block of 32 keys ahead of the products; a
// workgroup is one wave, so nothing waits for a barrier.
#pragma once

#include "awq_attend.hpp"

namespace awq {

template <int D>
constexpr int wave_ring() { return 4 * 32 * Tile<D>::ROW; }  // bytes: keys and values of two blocks

// Wave number `wave`; its own ring of wave_ring<D>() bytes.
template <int D, int R, bool LIST>
__device__ __forceinline__ void attend_wave(const AttendArgs& a, const CacheArgs& c, const SeqArgs& s, const UnitArgs& units,
                                            const Partials& p, int wave, lds_char* ring) {
  using T = Tile<D>;
  constexpr int LOADS = T::LOADS, PER = LOADS < 4 ? LOADS : 4;
  constexpr int SLOT = 32 * T::ROW;  // keys, then values, of a block
  const int lane = threadIdx.x & 63, group = units.group;
  const float scale = a.scale * kLog2E;

  const int list_rows = row_blocks(units, 1), of_list = LIST ? list_blocks(units, a.count) : 0;
  const int per_token = c.heads * list_rows * of_list;
  const Units n = LIST ? share_units(s.T * per_token) : count_units(s, units);
  int at = wave * n.each;
  const int end = min(n.total, at + n.each);

  const Sources<D> kept(lane);
  const Addresses<D, R> places((uint32_t)(uintptr_t)ring, lane);

  while (at < end) {
    // the segment that unit `at` is in
    Sequence seq{0, 0, 0, 0};
    int nth, blocks, key0 = 0, count = 0;  // nth: of the sequence's units
    const int* list = nullptr;
    if constexpr (LIST) {
      const int t = at / per_token;
      nth = at - t * per_token;
      blocks = of_list;
      const Sequence of = sequence_of(s, c.shift, t);
      if (of.rows == 0) {  // a row of no sequence
        at += per_token - nth;
        continue;
      }
      seq = Sequence{of.index, t, 1, t - of.row0 + of.place0() + 1};
    } else {
      int seen = 0;
      nth = 0;
      for (int b0 = 0; b0 < s.B; b0 += 64) {
        const Sequence q = sequence_at(s, c.shift, b0 + lane);
        const int mine = units_of(units, q), sum = seen + prefix_sum(mine);
        const unsigned long long owner = __ballot(sum > at && sum - mine <= at);
        if (owner != 0) {
          const int l = __builtin_ctzll(owner);
          seq = pick(q, l);
          nth = at - __builtin_amdgcn_readlane(sum - mine, l);
          break;
        }
        seen = __builtin_amdgcn_readlane(sum, 63);
      }
      if (seq.rows == 0) return;  // (some sequence holds it, at < total, unless the numbers changed meanwhile)
      blocks = key_blocks(units, seq.length);
      key0 = a.shared;
    }
    const int which = nth / blocks, block0 = nth - which * blocks;
    const int row_block = which / c.heads, head = which - row_block * c.heads;
    const int here = min(blocks - block0, end - at);
    at += here;
    const Rows rows{R * row_block, seq.rows * group, seq.row0, seq.place0()};
    // places of the rows: their own, and the least and greatest of them
    const int mine = (min(rows.first + (lane & (R - 1)), rows.total - 1)) / group;
    const int place = rows.place0 + mine, least = rows.place0 + rows.first / group;
    const int most = rows.place0 + (min(rows.first + R, rows.total) - 1) / group;
    if constexpr (LIST) {
      list = a.list + ((int64_t)seq.row0 * c.heads + head) * a.count;
      count = a.count;
    }
    Entries pages{s.tables + (int64_t)seq.index * s.width, list, count, s.width, head, 0, 0, 0, 0};

    Queries<D, R> q;
    read_queries(q, a, rows, group, head);
    Gathered<D, R> g;
    g.clear();

    int place0 = 0, place1 = 0, next0 = 0, next1 = 0;  // of the first of 16 keys
    auto load = [&](int block, lds_char* to) __attribute__((always_inline)) {
      const int key = key0 + 32 * (block0 + block);
      if (block == 0 || ((key + 16) >> c.shift) - pages.first >= 64) pages.read(c, key >> c.shift);
      Sources<D> from_lane = kept;
      asm volatile("" : "+v"(from_lane.keys[0]), "+v"(from_lane.values[0]));  // (each load's is formed here, not kept)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Keys16 from = keys16(pages, c, key + 16 * h);
        (h ? next1 : next0) = from.place;
        each<0, LOADS, PER>([&](auto ic) __attribute__((always_inline)) {
          constexpr int i = decltype(ic)::value;
          uint32_t k[PER], v[PER];
#pragma unroll
          for (int n = 0; n < PER; ++n) {
            k[n] = from_lane.key(i + n);
            v[n] = from_lane.value(i + n);
          }
          load_to_lds<PER>(reinterpret_cast<const char*>(c.k + from.at * D), k, to + 16 * h * T::ROW + 1024 * i);
          load_to_lds<PER>(reinterpret_cast<const char*>(c.v + from.at * D), v, to + SLOT + 16 * h * T::ROW + 1024 * i);
        });
      }
    };
    auto step = [&](int block, auto parity) __attribute__((always_inline)) {
      constexpr int HERE = 2 * SLOT * decltype(parity)::value, NEXT = 2 * SLOT - HERE;
      place0 = next0;
      place1 = next1;
      if (block + 1 < here) {
        load(block + 1, ring + NEXT);
        wait_loads<4 * LOADS>();
      } else {
        wait_loads<0>();
      }
      const Seen seen{place - place0, place - place1, least - place0 >= 15 && least - place1 >= 15};
      uint32_t strange = 0;
      if (!seen.all) {
        const uint64_t met = hide_strange<D, 32>(ring + HERE + SLOT, lane, 64, [&](int h, int& behind, int& upto) {
          behind = least - (h ? place1 : place0);
          upto = most - (h ? place1 : place0);
        });
        if (__any(met != 0)) {
          strange = (uint32_t)met;
          for (int m = 1; m < 64; m <<= 1) strange |= (uint32_t)__shfl_xor((int)strange, m);
          strange = __builtin_amdgcn_readfirstlane(strange);
        }
      }
      const Weights<R> p = attend_block<D, R, HERE, HERE + SLOT>(places, q, scale, seen, g);
      if (__builtin_expect(strange != 0, 0))
        gather_strange<D, R>(strange, p, seen, [&](int k) {
          const int key = key0 + 32 * (block0 + block) + k;
          const int page = list ? list[key >> c.shift] : key >> c.shift;
          const int64_t number = page_number(c, pages.table[page]);
          return c.v + (((number * c.heads + head) << c.shift) + (key & ((1 << c.shift) - 1))) * D;
        }, g);
    };
    load(0, ring);
    for (int block = 0; block < here; block += 2) {
      step(block, std::integral_constant<int, 0>{});
      if (block + 1 < here) step(block + 1, std::integral_constant<int, 1>{});
    }
    const bool whole = here == blocks;
    const int64_t slot = 2 * (int64_t)wave + (block0 > 0 ? 0 : 1);
    write_rows(g, a, p, rows, group, head, a.shared > 0 ? 0 : -1,
               whole ? nullptr : p.wave_stat + slot * 32, p.wave_sums + slot * 32 * D);
  }
}

}  // namespace awq
