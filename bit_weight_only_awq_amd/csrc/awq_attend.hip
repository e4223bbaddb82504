// Attention over a paged cache (awq_attend, awq_attend_pages): which kernels a
// batch takes, and the launch that joins parts.
//
// Few rows per sequence go to independent waves (awq_attend_waves.hip), many to
// workgroups of 128 rows (awq_attend_tiles.hip); shared keys to whichever suits the
// rows of all sequences together.
//
// Joining: with m the greatest of the parts' maxima, y = sum_i 2^(m_i - m) o_i / sum_i
// 2^(m_i - m) l_i over the parts, in a fixed order, in fp32.
#include "awq_attend.hpp"

namespace awq {
namespace {

struct JoinArgs {
  UnitArgs units;
  bool own_few;
  int own_slices, shared_slices;
};

// The join of some parts of one row, four channels per lane.
struct Joined {
  float4_t sums;
  float top, sum;
  __device__ __forceinline__ void add(float part_top, float part_sum, float4_t part) {
    if (part_top == -INFINITY && part_sum == 0.0f) return;  // (a part that saw no key)
    const float m = fmaxf(top, part_top);
    const float was = top == m ? 1.0f : __builtin_amdgcn_exp2f(top - m);
    const float is = part_top == m ? 1.0f : __builtin_amdgcn_exp2f(part_top - m);
    top = m;
    sum = sum * was + part_sum * is;
    sums = sums * was + part * is;
  }
};

// A row (token and query head) for WAVES waves; in a wave, LANES lanes hold the
// row's channels and 64 / LANES groups of them share the parts.
template <int D, int WAVES>
__global__ __launch_bounds__(256) void join_kernel(AttendArgs a, CacheArgs c, SeqArgs s, JoinArgs j, Partials p) {
  constexpr int LANES = D <= 64 ? 16 : D <= 128 ? 32 : 64, PARTS = 64 / LANES * WAVES;
  __shared__ float4_t sums[4][64];
  __shared__ float2 stats[4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * (4 / WAVES) + wave / WAVES;  // (every wave of the workgroup has one)
  const int t = (int)(row / a.q_heads), at = (int)(row - (int64_t)t * a.q_heads);
  const int group = j.units.group, head = at / group, channel = 4 * (lane & (LANES - 1));
  const int part = wave % WAVES * (64 / LANES) + lane / LANES;
  const bool live = channel < D && t < s.T;
  Joined x{float4_t(0.0f), -INFINITY, 0.0f};

  // the row's sequence and, among the waves' units, the first of it
  Sequence seq{0, 0, 0, 0};
  long long first = 0;
  Units n{0, 0, 1};
  if (j.own_few && !a.list) {
    n = count_units(s, j.units);
    long long seen = n.shared;
    for (int b0 = 0; b0 < s.B; b0 += 64) {
      const Sequence q = sequence_at(s, c.shift, b0 + lane);
      const long long mine = units_of(j.units, q), sum = seen + prefix_sum64(mine);
      const unsigned long long owner = __ballot(t >= q.row0 && t < q.row0 + q.rows);
      if (owner != 0) {
        const int l = __builtin_ctzll(owner);
        seq = pick(q, l);
        first = lane64(sum - mine, l);
        break;
      }
      seen = lane64(sum, 63);
    }
  } else {
    seq = sequence_of(s, c.shift, t);
  }
  bool write = seq.rows > 0;
  if (seq.rows > 0 && t - seq.row0 + seq.place0() >= 0) {
    auto slice = [&](int i) __attribute__((always_inline)) {
      const int64_t from = i * p.rows + row;
      const float2 stat = p.stat[from];
      x.add(stat.x, stat.y, *reinterpret_cast<const float4_t*>(p.sums + from * D + channel));
    };
    // the waves' pieces of the segment that begins at `unit`, row r of its 32; whole, it is in slice `whole`, or in y
    auto pieces = [&](long long unit, int blocks, int r, int whole) __attribute__((always_inline)) {
      const int w0 = (int)(unit / n.each), w1 = (int)((unit + blocks - 1) / n.each);
      if (w0 == w1) {
        if (whole < 0) write = false;
        else if (live && part == 0) slice(whole);
        return;
      }
      if (live)
        for (int w = w0 + part; w <= w1; w += PARTS) {
          const int64_t from = (2 * (int64_t)w + ((long long)w * n.each > unit ? 0 : 1)) * 32 + r;
          const float2 stat = p.wave_stat[from];
          x.add(stat.x, stat.y, *reinterpret_cast<const float4_t*>(p.wave_sums + from * D + channel));
        }
    };
    if (a.list) {
      const int list_rows = row_blocks(j.units, 1), r = at - head * group, blocks = ((a.count << c.shift) + 31) >> 5;
      const long long all = (long long)s.T * c.heads * list_rows * blocks;
      n.each = (int)max((all + j.units.waves - 1) / j.units.waves, (long long)j.units.least);
      pieces((((long long)t * list_rows + (r >> 5)) * c.heads + head) * blocks, blocks, r & 31, -1);
    } else if (j.own_few) {
      const int r = (t - seq.row0) * group + at - head * group, blocks = key_blocks(j.units, seq.length);
      pieces(first + ((long long)(r >> 5) * c.heads + head) * blocks, blocks, r & 31, j.own_slices > 0 ? 0 : -1);
    }
    if (j.units.shared) {
      const int r = (t - all_rows(s, 0).row0) * group + at - head * group, blocks = (j.units.shared_keys + 31) >> 5;
      pieces(((long long)(r >> 5) * c.heads + head) * blocks, blocks, r & 31, 1);
    }
    // what workgroups of 128 rows made
    if (live) {
      const int from = j.own_few ? j.own_slices : 0, to = j.own_slices + (j.units.shared ? 0 : j.shared_slices);
      for (int i = from + part; i < to; i += PARTS) slice(i);
    }
  }
#pragma unroll
  for (int m = LANES; m < 64; m <<= 1) {
    float4_t other;
#pragma unroll
    for (int i = 0; i < 4; ++i) other[i] = __shfl_xor(x.sums[i], m);
    const float top = __shfl_xor(x.top, m), sum = __shfl_xor(x.sum, m);
    // (in the order of the lanes, so that both get the same)
    Joined lower = lane & m ? Joined{other, top, sum} : x;
    if (lane & m) lower.add(x.top, x.sum, x.sums);
    else lower.add(top, sum, other);
    x = lower;
  }
  if constexpr (WAVES > 1) {
    sums[wave][lane] = x.sums;
    if (lane == 0) stats[wave] = float2{x.top, x.sum};
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 1; w < WAVES; ++w) x.add(stats[w].x, stats[w].y, sums[w][lane]);
  }
  if (!write || !live || lane >= LANES) return;
  const float by = x.sum == 0.0f ? 0.0f : 1.0f / x.sum;
  half4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (_Float16)(x.sum == 0.0f ? 0.0f : x.sums[i] * by);
  *reinterpret_cast<half4_t*>(a.y + t * a.ldy + (int64_t)at * D + channel) = v;
}

constexpr int kUnits = 256;  // compute units

// The keys' splits over which `tiles` workgroups take the least time, in rounds of two per compute unit (one where
// a head is 256 wide), a stage being the unit and what a workgroup does besides costing `extra` of them.
int splits_of(int64_t tiles, int64_t stages, int slots, double extra) {
  int best = 1;
  double least = 1e300;
  for (int n = 1; n <= 64 && n * 2 <= stages + 1; ++n) {
    const double rounds = (double)((tiles * n + slots - 1) / slots);
    const double time = rounds * ((double)((stages + n - 1) / n) + extra) + 0.3 * n;
    if (time < least) {
      least = time;
      best = n;
    }
  }
  return best;
}

AttendPlan plan_of(int T, int B, int q_heads, int kv_heads, int dim, int page_size, int width, int shared, bool list) {
  const int group = q_heads / kv_heads, stage = dim == 256 ? 32 : 64, slots = dim == 256 ? kUnits : 2 * kUnits;
  const int64_t rows = (int64_t)T * group;
  AttendPlan p{};
  p.own_few = list || rows <= 32 * (int64_t)B;
  p.prefix = shared == 0 ? 0 : p.own_few && rows <= 32 ? 1 : 2;
  p.waves = kUnits * (dim == 256 ? 2 : dim == 128 ? 5 : 6);
  p.least = 2;
  p.own_splits = p.prefix_splits = 1;
  if (p.prefix == 2) p.prefix_splits = splits_of((rows + 127) / 128 * kv_heads, (shared + stage - 1) / stage, slots, 3.0);
  if (!p.own_few) {
    const int64_t keys = (int64_t)width * page_size - shared;
    p.own_splits = splits_of(((rows + 127) / 128 + B / 2) * kv_heads, (keys + stage - 1) / stage, slots, 3.0);
  }
  return p;
}

template <int D>
void launch_join(const AttendArgs& a, const CacheArgs& c, const SeqArgs& s, const JoinArgs& j, const Partials& p,
                 hipStream_t stream) {
  const int64_t rows = (int64_t)s.T * a.q_heads;
  if (j.own_few) hipLaunchKernelGGL((join_kernel<D, 4>), dim3((unsigned)rows), dim3(256), 0, stream, a, c, s, j, p);
  else hipLaunchKernelGGL((join_kernel<D, 1>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream, a, c, s, j, p);
}

}  // namespace

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
  if (plan.prefix == 2 || !plan.own_few) e = launch_attend_tiles(a, c, s, plan, p, stream);
  if (e == hipSuccess && plan.own_few) e = launch_attend_waves(a, c, s, plan, p, stream);
  if (e != hipSuccess || (!plan.own_few && plan.slices() == 0)) return e;
  const JoinArgs j{unit_args(a, c, plan), plan.own_few, plan.own_slices(), plan.slices() - plan.own_slices()};
  if (c.dim == 64) launch_join<64>(a, c, s, j, p, stream);
  else if (c.dim == 96) launch_join<96>(a, c, s, j, p, stream);
  else if (c.dim == 128) launch_join<128>(a, c, s, j, p, stream);
  else launch_join<256>(a, c, s, j, p, stream);
  return hipGetLastError();
}

}  // namespace awq
