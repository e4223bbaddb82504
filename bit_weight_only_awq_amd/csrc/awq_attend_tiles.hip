// Attention of many rows (prompts, and the shared keys of a batch): workgroups of
// 128 rows, four waves of 32, that share each stage of keys and values.
//
// Mathematics: awq_attend_block.hpp's.  A row is a token and a query head of one key
// head, so the query heads of a group and, for the shared keys, the sequences of the
// batch are rows of one product: the shared keys are read once per 128 rows, not
// once per sequence.
//
// Bound: the matrix cores (4 D operations per row and key) beside the
// exponentials.  A stage of keys and values goes straight to LDS while the one
// before it is multiplied, with one barrier per stage.  Where the row tiles are
// too few for the chip, the keys are split as well and the parts joined by a second
// launch.
#include "awq_attend.hpp"

namespace awq {
namespace {

constexpr int kTile = 128;  // rows of a workgroup

// `shared_tiles` workgroup rows of the shared keys first, then the sequences' own.
struct TileArgs {
  int group, shared_tiles, shared_splits, own_tiles, own_splits, own_slice, shared_slice;
  int descending;  // of the own tiles (per key head and split), those that come first, from the last rows up
};

template <int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attend_tiles_kernel(AttendArgs a, CacheArgs c, SeqArgs s, TileArgs x,
                                                                             Partials p) {
  using T = Tile<D>;
  constexpr int KEYS = D == 256 ? 32 : 64;                  // of a stage
  constexpr int LOADS = KEYS / 16 * T::LOADS / 4;           // of a wave and stage, of keys and of values each
  constexpr int SLOT = KEYS * T::ROW;
  __shared__ __attribute__((aligned(1024))) char ring[4 * SLOT];  // keys, then values, of two stages
  __shared__ __attribute__((aligned(1024))) char queries[Queries<D>::BYTES ? 4 * Queries<D>::BYTES : 16];
  __shared__ uint32_t strange[2][2];  // of a stage and the next
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), group = x.group;
  const float scale = a.scale * kLog2E;

  // the tile: key heads next to each other (one XCD keeps meeting the same); the last rows, which have the most keys,
  // first, and where there are at most two workgroups per compute unit the second ones the other way around, so that
  // each unit gets one with many keys and one with few
  const int head = blockIdx.x % c.heads;
  int nth = blockIdx.x / c.heads;
  const bool shared = nth < x.shared_tiles * x.shared_splits;
  int split, splits, slice, key0, keys;
  Rows32 rows;  // of the workgroup, then of the wave
  Sequence seq;
  if (shared) {
    split = nth / x.shared_tiles;
    splits = x.shared_splits;
    slice = x.shared_slice + split;
    seq = all_rows(s, a.shared);
    rows = Rows32{kTile * (nth - split * x.shared_tiles), seq.rows * group, seq.row0, 0};
    if (rows.first >= rows.total) return;
    key0 = 0;
    keys = a.shared;
  } else {
    nth -= x.shared_tiles * x.shared_splits;
    split = nth / x.own_tiles;
    splits = x.own_splits;
    slice = x.own_slice < 0 ? -1 : x.own_slice + split;
    const int turn = nth - split * x.own_tiles, wanted = turn < x.descending ? x.own_tiles - 1 - turn : turn - x.descending;
    int seen = 0;
    bool found = false;
    for (int b0 = 0; b0 < s.B; b0 += 64) {
      const Sequence q = sequence_at(s, c.shift, b0 + lane);
      const int tiles = (q.rows * group + kTile - 1) / kTile, sum = seen + prefix_sum(tiles);
      const unsigned long long owner = __ballot(sum > wanted && sum - tiles <= wanted);
      if (owner != 0) {
        const int l = __builtin_ctzll(owner);
        seq = pick(q, l);
        rows = Rows32{kTile * (wanted - __builtin_amdgcn_readlane(sum - tiles, l)), seq.rows * group, seq.row0, seq.place0()};
        found = true;
        break;
      }
      seen = __builtin_amdgcn_readlane(sum, 63);
    }
    if (!found) return;
    key0 = a.shared;
    keys = rows.place0 + (min(rows.first + kTile, rows.total) - 1) / group + 1 - key0;
  }
  const int stages = keys > 0 ? (keys + KEYS - 1) / KEYS : 0;
  const int from = (int)((long long)stages * split / splits), to = (int)((long long)stages * (split + 1) / splits);

  // least and greatest place of the workgroup's rows, then of the wave's
  const int tile_least = shared ? a.shared - 1 : rows.place0 + rows.first / group;
  const int tile_most = key0 + keys - 1;
  if (threadIdx.x < 4) strange[threadIdx.x >> 1][threadIdx.x & 1] = 0;
  rows.first += 32 * wave;
  const bool live = rows.first < rows.total;
  const int mine = min(rows.first + (lane & 31), rows.total - 1) / group;
  const int place = shared ? a.shared - 1 : rows.place0 + mine;
  const int least = shared ? a.shared - 1 : rows.place0 + min(rows.first, rows.total - 1) / group;
  const int most = !live ? -1 : shared ? a.shared - 1 : rows.place0 + (min(rows.first + 32, rows.total) - 1) / group;

  Queries<D> q;
  q.place((lds_char*)queries + wave * Queries<D>::BYTES);
  read_queries(q, a, rows, group, head);
  Gathered<D> g;
  g.clear();

  // this wave's loads of a stage: LOADS of keys and of values, all from one group of 16 keys
  constexpr int PER = T::LOADS / LOADS;  // waves per 16 keys
  static_assert(T::LOADS % LOADS == 0, "a wave's loads are of one group of keys");
  const int sixteen = wave / PER, part = wave % PER;
  const Sources<D> kept(lane, part * LOADS);
  const Addresses<D> places((uint32_t)(uintptr_t)(lds_char*)ring, lane);
  Entries pages{s.tables + (int64_t)seq.index * s.width, nullptr, 0, s.width, 0, 0, 0};
  auto load = [&](int stage, lds_char* slot) __attribute__((always_inline)) {
    const int key = key0 + KEYS * stage;
    if (stage == from || ((key + KEYS - 16) >> c.shift) - pages.first >= 64) pages.read(c, key >> c.shift);
    const Keys16 source = keys16(pages, c, head, key + 16 * sixteen);
    const char* k = reinterpret_cast<const char*>(c.k + source.at * D);
    const char* v = reinterpret_cast<const char*>(c.v + source.at * D);
    Sources<D> from_lane = kept;
    asm volatile("" : "+v"(from_lane.keys[0]), "+v"(from_lane.values[0]));  // (each load's is formed here, not kept)
    lds_char* to = slot + 16 * sixteen * T::ROW + 1024 * part * LOADS;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) load_to_lds(k + from_lane.key(i), to + 1024 * i);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) load_to_lds(v + from_lane.value(i), to + SLOT + 1024 * i);
  };
  auto step = [&](int stage, auto parity) __attribute__((always_inline)) {
    constexpr int HERE = 2 * SLOT * decltype(parity)::value, NEXT = 2 * SLOT - HERE;
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (stage + 1 < to) load(stage + 1, (lds_char*)ring + NEXT);
    // past the least place of the workgroup's rows some values are not to be seen by some row
    const int key = key0 + KEYS * stage;
    const bool ragged = key + KEYS - 1 > tile_least;
    if (ragged) {
      const uint64_t met = hide_strange<D, KEYS>((lds_char*)ring + HERE + SLOT, threadIdx.x, 256, [&](int h, int& behind, int& upto) {
        behind = tile_least - key - 16 * h;
        upto = tile_most - key - 16 * h;
      });
      if ((uint32_t)met) atomicOr(&strange[stage & 1][0], (uint32_t)met);
      if (met >> 32) atomicOr(&strange[stage & 1][1], (uint32_t)(met >> 32));
      if (threadIdx.x < 2) strange[(stage + 1) & 1][threadIdx.x] = 0;
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    }
    each<0, KEYS / 32, 1>([&](auto bc) __attribute__((always_inline)) {
      constexpr int b = decltype(bc)::value;
      const int first = key + 32 * b;
      if (first > most) return;
      const Seen seen{place - first, place - first - 16, least - first >= 31};
      const uint32_t odd = ragged ? __builtin_amdgcn_readfirstlane(strange[stage & 1][b]) : 0;
      attend_block<D, HERE + 32 * b * T::ROW, HERE + SLOT + 32 * b * T::ROW>(places, q, scale, seen, odd, [&](int k) {
        const int64_t number = page_number(c, pages.table[(first + k) >> c.shift]);
        return c.v + (((number * c.heads + head) << c.shift) + ((first + k) & ((1 << c.shift) - 1))) * D;
      }, g);
    });
  };
  if (from < to) load(from, (lds_char*)ring);
  for (int stage = from; stage < to; stage += 2) {
    step(stage, std::integral_constant<int, 0>{});
    if (stage + 1 < to) step(stage + 1, std::integral_constant<int, 1>{});
  }
  if (live) write_rows(g, scale, a, p, rows, group, head, slice, nullptr, nullptr);
}

template <int D>
void launch(const AttendArgs& a, const CacheArgs& c, const SeqArgs& s, const TileArgs& x, const Partials& p,
            hipStream_t stream) {
  const unsigned grid = (unsigned)((x.shared_tiles * x.shared_splits + x.own_tiles * x.own_splits) * c.heads);
  hipLaunchKernelGGL((attend_tiles_kernel<D>), dim3(grid), dim3(256), 0, stream, a, c, s, x, p);
}

}  // namespace

hipError_t launch_attend_tiles(const AttendArgs& a, const CacheArgs& c, const SeqArgs& s, const AttendPlan& plan,
                               const Partials& p, hipStream_t stream) {
  const int group = a.q_heads / c.heads;
  const int64_t rows = (int64_t)s.T * group, most = rows / kTile + s.B;  // (a ragged tile per sequence at most)
  TileArgs x{group, 0, 1, 0, 1, plan.own_slices() > 0 ? 0 : -1, plan.own_slices(), 0};
  if (plan.prefix == 2) {
    x.shared_tiles = (int)((rows + kTile - 1) / kTile);
    x.shared_splits = plan.prefix_splits;
  }
  if (!plan.own_few) {
    x.own_tiles = (int)(most < rows ? most : rows);
    x.own_splits = plan.own_splits;
    const int first = (kUnits + c.heads - 1) / c.heads;
    const bool twice = x.shared_tiles == 0 && x.own_splits == 1 && x.own_tiles > first && x.own_tiles <= 2 * first;
    x.descending = twice && c.dim < 256 ? first : x.own_tiles;
  }
  if (c.dim == 64) launch<64>(a, c, s, x, p, stream);
  else if (c.dim == 96) launch<96>(a, c, s, x, p, stream);
  else if (c.dim == 128) launch<128>(a, c, s, x, p, stream);
  else launch<256>(a, c, s, x, p, stream);
  return hipGetLastError();
}

}  // namespace awq
