// Attention over a paged cache (awq_attend, awq_attend_pages): which kernels a
// batch takes, and the launch that joins parts.
//
// Few rows per sequence go to independent waves (awq_attend_waves.hip), many to
// workgroups of 128 rows (awq_attend_tiles.hip), and shared keys to these, with the
// rows of all sequences together.
//
// Joining: with m the greatest of the parts' maxima, y = sum_i 2^((m_i - m) c) o_i / sum_i
// 2^((m_i - m) c) l_i over the parts, in a fixed order, in fp32.  Bound: a launch and the
// chain offsets -> which parts -> parts (4.6-6.7 us); 16 to 30 MB of parts of many rows
// 14 us.
#include "awq_attend.hpp"

namespace awq {
namespace {

struct JoinArgs {
  UnitArgs units;
  int slices;  // the own keys' (where there are shared keys) and theirs
};

// Where waves made the parts of the own keys: a wave per row (token and query
// head), 64 parts at a time, a lane holding each part's maximum and sum, then LANES
// lanes their share of the channels and 64 / LANES groups of lanes every such part.
template <int D>
__global__ __launch_bounds__(256) void join_kernel(AttendArgs a, CacheArgs c, SeqArgs s, JoinArgs j, Partials p) {
  constexpr int LANES = D <= 64 ? 16 : D <= 128 ? 32 : 64, GROUPS = 64 / LANES, AHEAD = 8;
  const int lane = threadIdx.x & 63;
  const int row = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int t = row / a.q_heads, at = row - t * a.q_heads;
  if (t >= s.T) return;
  const int group = j.units.group, head = at / group, g = at - head * group;

  // the row's sequence and, among the waves' units, the first of it
  Sequence seq{0, 0, 0, 0};
  int first = 0;
  Units n{0, 1};
  if (!a.list) {
    int seen = 0;
    for (int b0 = 0; b0 < s.B; b0 += 64) {
      const Sequence q = sequence_at(s, c.shift, b0 + lane);
      const int mine = units_of(j.units, q), sum = seen + prefix_sum(mine);
      const unsigned long long owner = __ballot(t >= q.row0 && t < q.row0 + q.rows);
      if (owner != 0 && seq.rows == 0) {
        const int l = __builtin_ctzll(owner);
        seq = pick(q, l);
        first = __builtin_amdgcn_readlane(sum - mine, l);
      }
      seen = __builtin_amdgcn_readlane(sum, 63);
    }
    n = share_units(seen);
  } else {
    seq = sequence_of(s, c.shift, t);
    n = share_units(s.T * c.heads * row_blocks(j.units, 1) * list_blocks(j.units, a.count));
  }
  if (seq.rows == 0) return;  // a row of no sequence stays as it is

  // The row's parts: `pieces` of waves from `wave0` on, then slices: slice 0, the own keys, if a wave had them all, and the
  // shared keys'.  (A row without a place has parts as well: those of its own keys, all empty, and those of shared
  // keys, not its.)
  const bool placed = t - seq.row0 + seq.place0() >= 0;
  const int blocks = a.list ? list_blocks(j.units, a.count) : key_blocks(j.units, seq.length);
  const int r = a.list ? g : (t - seq.row0) * group + g, nth = r / j.units.rows, own_row = r - nth * j.units.rows;
  const int unit = first + (((a.list ? t * row_blocks(j.units, 1) : 0) + nth) * c.heads + head) * blocks;
  // (within the waves that there are, also where sequences overlap and the units are too many to count)
  const int wave0 = min(max(unit / n.each, 0), kWaves - 1);
  int pieces = min((unit + blocks - 1) / n.each, kWaves - 1) - wave0 + 1, slice0 = 1;
  if (pieces == 1) {
    if (j.slices == 0) return;  // the result is in place
    pieces = slice0 = 0;
  }
  const int parts = placed ? pieces + max(j.slices - slice0, 0) : 0;

  float4_t sums = float4_t(0.0f);
  const float c2 = a.scale * kLog2E;
  float top = -INFINITY, total = 0.0f;
  const int channel = 4 * (lane & (LANES - 1));
  const bool live = channel < D;
  for (int i0 = 0; i0 < parts; i0 += 64) {
    // where part i0 + lane is: a number of 32 rows of a wave, negative, or of a row of a slice
    int i = i0 + lane, from = 0;
    float2 stat{-INFINITY, 0.0f};
    if (i < parts) {
      if (i < pieces) {
        const int w = wave0 + i;
        from = -1 - ((2 * w + (w * n.each > unit ? 0 : 1)) * 32 + own_row);
        stat = p.wave_stat[-1 - from];
      } else {
        from = (int)((slice0 + i - pieces) * p.rows) + row;
        stat = p.stat[from];
      }
    }
    // (the first values are on their way while the maxima are compared, and the next while some are added)
    const int here = min(64, parts - i0);
    float4_t v[AHEAD];
    const auto load = [&](int k0) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int of = k0 + k * GROUPS + lane / LANES, where = __shfl(from, of & 63);
        v[k] = float4_t(0.0f);
        if (of < here && live)
          v[k] = *reinterpret_cast<const float4_t*>(
              (where < 0 ? p.wave_sums + (int64_t)(-1 - where) * D : p.sums + (int64_t)where * D) + channel);
      }
    };
    load(0);
    float m = stat.x;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
    m = fmaxf(m, top);
    // (a part that saw no key counts nothing, also where none did)
    const float share = stat.x == -INFINITY && stat.y == 0.0f ? 0.0f : stat.x == m ? 1.0f : __builtin_amdgcn_exp2f((stat.x - m) * c2);
    float sum = share * stat.y;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x);
    const float carry = top == m ? 1.0f : __builtin_amdgcn_exp2f((top - m) * c2);
    total = total * carry + sum;
    if (i0 > 0) sums *= carry;
    top = m;
    for (int k0 = 0; k0 < here; k0 += AHEAD * GROUPS) {
      float4_t w[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) w[k] = v[k];
      if (k0 + AHEAD * GROUPS < here) load(k0 + AHEAD * GROUPS);
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int of = k0 + k * GROUPS + lane / LANES;
        const float by = __shfl(share, of & 63);
        sums += w[k] * (of < here ? by : 0.0f);
      }
    }
  }
#pragma unroll
  for (int m = LANES; m < 64; m <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[i] += __shfl_xor(sums[i], m);
  if (!live || lane >= LANES) return;
  const float by = total == 0.0f ? 0.0f : 1.0f / total;
  half4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (_Float16)(total == 0.0f ? 0.0f : sums[i] * by);
  *reinterpret_cast<half4_t*>(a.y + t * a.ldy + (int64_t)at * D + channel) = v;
}

// The same where all parts are slices (workgroups of 128 rows made them): LANES
// lanes per row, nothing to look up but whether the row is of a sequence at all.
template <int D>
__global__ __launch_bounds__(256) void join_slices_kernel(AttendArgs a, SeqArgs s, int slices, Partials p) {
  constexpr int LANES = D <= 64 ? 16 : D <= 128 ? 32 : 64, AHEAD = 4;
  const int row = (int)(blockIdx.x * (256 / LANES) + threadIdx.x / LANES), channel = 4 * (threadIdx.x & (LANES - 1));
  const int t = row / a.q_heads, at = row - t * a.q_heads;
  if (t < s.offsets[0] || t >= min(s.offsets[s.B], s.T) || channel >= D) return;
  float4_t sums = float4_t(0.0f);
  const float c2 = a.scale * kLog2E;
  float top = -INFINITY, total = 0.0f;
  bool placed = true;
  float2 next_stat[AHEAD];
  float4_t next_part[AHEAD];
  const auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {  // (past the last slice: the last again, counted as nothing)
      const int64_t from = min(i0 + i, slices - 1) * p.rows + row;
      next_stat[i] = p.stat[from];
      next_part[i] = *reinterpret_cast<const float4_t*>(p.sums + from * D + channel);
    }
  };
  load(0);
  for (int i0 = 0; i0 < slices; i0 += AHEAD) {
    float2 stat[AHEAD];
    float4_t part[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) stat[i] = next_stat[i], part[i] = next_part[i];
    if (i0 + AHEAD < slices) load(i0 + AHEAD);
    float m = top;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      placed = placed && stat[i].y != kNoPlace;
      m = fmaxf(m, stat[i].x);
    }
    const float carry = top == m ? 1.0f : __builtin_amdgcn_exp2f((top - m) * c2);
    total *= carry;
    sums *= carry;
    top = m;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (i0 + i >= slices || (stat[i].x == -INFINITY && stat[i].y == 0.0f)) continue;
      const float share = stat[i].x == m ? 1.0f : __builtin_amdgcn_exp2f((stat[i].x - m) * c2);
      total += stat[i].y * share;
      sums += part[i] * share;
    }
  }
  const bool none = total == 0.0f || !placed;
  const float by = 1.0f / total;
  half4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (_Float16)(none ? 0.0f : sums[i] * by);
  *reinterpret_cast<half4_t*>(a.y + t * a.ldy + (int64_t)at * D + channel) = v;
}

// The keys' splits over which `tiles` workgroups take the least time, in rounds of two per compute unit (one where
// a head is 256 wide), a stage being the unit, what a workgroup does besides costing three of them, and writing and
// reading the parts of a tile 0.0085 (128 rows of fp32 sums, there and back).  (Both costs are those of heads of 128
// channels, taken for the others too.)
int splits_of(int64_t tiles, int64_t stages, int slots) {
  int best = 1;
  double least = 1e300;
  for (int n = 1; n <= 64 && n * 2 <= stages + 1 && (n == 1 || tiles * n <= 16 * slots); ++n) {
    const double rounds = (double)((tiles * n + slots - 1) / slots);
    const double time = rounds * ((double)((stages + n - 1) / n) + 3.0) + (n > 1 ? 0.0085 * n * tiles : 0.0);
    if (time < least) {
      least = time;
      best = n;
    }
  }
  return best;
}

// Which kernels, measured on both sides (us; sequences x new tokens x query heads of a key head):
// Up to 32 rows per sequence on average (a row: a token and a query head of one key head) the waves, which share ragged
// batches out evenly; past that they would read the keys twice.  Waves, row tiles, with as many tokens before each
// sequence / with 7 to twice as many:
//   8 x 1 x 8, 4000     35.2, 38.0 / 41.3, 48.2     16 x 1 x 4, 3000   45.1, 48.4 / 52.9, 62.3
//   8 x 4 x 8           39.7, 42.2 / 46.7, 52.2     16 x 8 x 4         52.2, 53.5 / 61.0, 66.5
//   8 x 8 x 8 (tiles)   57.4, 44.6 / 65.1, 52.1     16 x 16 x 4 (tiles)  75.1, 52.6 / 92.8, 70.4
//   20 x 8 x 3, 2000    45.5, 46.2 / 50.6, 56.8     20 x 16 x 3 (tiles)  69.4, 46.5 / 78.8, 60.0
//   30 x 1 x 1, 1000    96.4, 95.6 / 119, 120       30 x 8 x 1         105, 97 / 134, 125
//   30 x 4 x 1          99.5, 96.1 / 123, 123       30 x 32 x 1        135, 105 / 169, 135
// So for a single query head per key head (the last two lines) the rule is off: from about four tokens on the join of
// their many rows costs more than the waves save, up to 29 %.
// Up to 16 rows the waves' products are of 16: 8 x 2 x 8 32.0, of 32 32.4; 8 x 4 x 8 43.1, 33.9.
// Shared keys always by row tiles: 1 x 1 x 8 after 8192 19.0, by waves 30.9; 16 x 1 x 8 26.1, 61.4; and in one launch with
// the waves, whose products are of 16 rows there: 16 x 1 x 8 25.9, in two 38.2; 61 x 1 x 8 47, 68; 1 x 6 x 3 after 1600 18, 23;
// 61 x 1 x 8 with heads of 64: 30, 47, of 96: 36, 56, of 256, where row tiles begin as the waves end: 99, 104.
AttendPlan plan_of(int T, int B, int q_heads, int kv_heads, int dim, int page_size, int width, int shared, bool list) {
  const int group = q_heads / kv_heads, stage = dim == 256 ? 32 : 64, slots = dim == 256 ? kUnits : 2 * kUnits;
  const int64_t rows = (int64_t)T * group;
  AttendPlan p{};
  p.shared = shared > 0;
  // (units of the waves: 16 rows, at least a block of them per sequence, times key heads and blocks of 32 keys)
  const int64_t units = kv_heads * (rows / 16 + B) * ((int64_t)width * page_size / 32 + 1);
  p.own_few = list || (rows <= 32 * (int64_t)B && units < kMostUnits);
  p.rows = p.shared || rows <= 16 * (int64_t)(list ? T : B) ? 16 : 32;
  p.own_splits = p.shared_splits = 1;
  if (p.shared)
    p.shared_splits = splits_of((rows + 127) / 128 * kv_heads, (shared + stage - 1) / stage, p.both() ? kUnits : slots);
  if (!p.own_few) {
    const int64_t keys = (int64_t)width * page_size - shared;
    p.own_splits = splits_of(((rows + 127) / 128 + B / 2) * kv_heads, (keys + stage - 1) / stage, slots);
  }
  return p;
}

template <int D>
void launch_join(const AttendArgs& a, const CacheArgs& c, const SeqArgs& s, bool own_few, const JoinArgs& j,
                 const Partials& p, hipStream_t stream) {
  const int64_t rows = (int64_t)s.T * a.q_heads;
  constexpr int ROWS = 256 / (D <= 64 ? 16 : D <= 128 ? 32 : 64);  // of a workgroup
  if (own_few)
    hipLaunchKernelGGL((join_kernel<D>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream, a, c, s, j, p);
  else
    hipLaunchKernelGGL((join_slices_kernel<D>), dim3((unsigned)((rows + ROWS - 1) / ROWS)), dim3(256), 0, stream, a, s,
                       j.slices, p);
}

}  // namespace

bool attend_fits(int T, int B, int q_heads, int kv_heads, int dim, int page_size, int width, int shared) {
  const AttendPlan p = plan_of(T, B, q_heads, kv_heads, dim, page_size, width, shared, false);
  const int64_t tiles = p.shared || !p.own_few ? tile_workgroups(tile_args(p, T, B, q_heads, kv_heads, dim), kv_heads) : 0;
  return (tiles + (p.both() ? kUnits : 0)) * 256 < (int64_t)1 << 32;
}
size_t attend_workspace_bytes(int T, int B, int q_heads, int kv_heads, int dim, int page_size, int width, int shared) {
  return partial_bytes(plan_of(T, B, q_heads, kv_heads, dim, page_size, width, shared, false), (int64_t)T * q_heads, dim);
}
size_t attend_list_workspace_bytes(int T, int q_heads, int kv_heads, int dim, int page_size, int count) {
  return partial_bytes(plan_of(T, 1, q_heads, kv_heads, dim, page_size, count, 0, true), (int64_t)T * q_heads, dim);
}

hipError_t launch_attend(const AttendArgs& a, const CacheArgs& c, const SeqArgs& s, void* workspace, hipStream_t stream) {
  const bool list = a.list != nullptr;
  const AttendPlan plan = plan_of(s.T, s.B, a.q_heads, c.heads, c.dim, 1 << c.shift, list ? a.count : s.width, a.shared, list);
  const Partials p = partials(plan, (int64_t)s.T * a.q_heads, c.dim, workspace);
  hipError_t e = hipSuccess;
  if (plan.shared || !plan.own_few) e = launch_attend_tiles(a, c, s, plan, p, stream);
  if (e == hipSuccess && plan.own_few && !plan.both()) e = launch_attend_waves(a, c, s, plan, p, stream);
  if (e != hipSuccess || (!plan.own_few && plan.slices() == 0)) return e;
  const JoinArgs j{unit_args(a, c, plan), plan.slices()};
#define AWQ_JOIN(D) launch_join<D>(a, c, s, plan.own_few, j, p, stream)
  if (c.dim == 64) AWQ_JOIN(64);
  else if (c.dim == 96) AWQ_JOIN(96);
  else if (c.dim == 128) AWQ_JOIN(128);
  else AWQ_JOIN(256);
#undef AWQ_JOIN
  return hipGetLastError();
}

}  // namespace awq
