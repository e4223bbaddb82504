// New tokens into a paged cache (awq_append_kv): the rows of a fused q/k/v layer,
// queries and keys rotated by their positions on the way, keys and values into
// their sequences' pages, and each touched page's lowest and highest key.
//
// Mathematics: pair i of a head's first `rotary` channels turns by the angle
// position * inv_freq[i]; (a, b) -> (a cos - b sin, b cos + a sin) in fp32, one
// rounding to fp16.  The angle is a product of 64 bits, reduced to a quarter turn
// in 64 bits as well, so that a position of a million is as exact as one of ten;
// sine and cosine of the rest (at most an eighth of a turn) are Taylor sums to
// 2e-9 and 3e-8.  A page's bounds are the channel-wise least and greatest of its
// stored (rounded) keys: exact, whatever the order, so appending a token at a time
// and a prompt at once leave the same bits.
//
// Bound: HBM for prompts (every row read and written once); for a few tokens the
// launch and the chain lengths -> table -> row.  One workgroup takes the new
// tokens of one page (so that nobody else writes its bounds) and one key head's
// keys and values, or kHeads query heads; the angles' sines and cosines are shared
// by the workgroup through LDS, 16 tokens at a time.
#include "awq_cache.hpp"

namespace awq {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;  // tokens whose sines and cosines are in LDS at a time
constexpr int kHeads = 4;    // query heads of a workgroup

struct Turn {
  float cos, sin;
};

__device__ __forceinline__ Turn turn_of(int position, float freq) {
  const double t = (double)position * (double)freq * 0.63661977236758134;  // in quarter turns: 2 / pi
  const double whole = __builtin_rint(t);
  const float x = (float)(t - whole) * 1.5707963267948966f, y = x * x;
  const float sin = x + x * y * (-1.6666666666666666e-1f + y * (8.3333333333333333e-3f + y * (-1.984126984126984e-4f +
                                                                                            y * 2.7557319223985893e-6f)));
  const float cos = 1.0f + y * (-0.5f + y * (4.1666666666666664e-2f + y * (-1.3888888888888889e-3f +
                                                                          y * 2.48015873015873e-5f)));
  const int quarter = (int)(long long)whole & 3;
  const float s = quarter & 1 ? cos : sin, c = quarter & 1 ? sin : cos;
  return Turn{quarter == 1 || quarter == 2 ? -c : c, quarter >= 2 ? -s : s};
}

// Sixteen channels of a head: two chunks of eight.  Unit u of the rotated
// part holds the pairs 8 u .. 8 u + 7.
struct Unit {
  int lo, hi;
};
__device__ __forceinline__ Unit unit_of(int u, int rotary, bool interleaved) {
  const bool apart = 16 * u < rotary && !interleaved;
  return apart ? Unit{8 * u, rotary / 2 + 8 * u} : Unit{16 * u, 16 * u + 8};
}

__device__ __forceinline__ void rotate(half8_t& a, half8_t& b, const Turn* turn, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Turn p = turn[i], q = turn[4 + i];
      const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
      a[2 * i] = (_Float16)(a0 * p.cos - a1 * p.sin);
      a[2 * i + 1] = (_Float16)(a1 * p.cos + a0 * p.sin);
      b[2 * i] = (_Float16)(b0 * q.cos - b1 * q.sin);
      b[2 * i + 1] = (_Float16)(b1 * q.cos + b0 * q.sin);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const Turn p = turn[i];
      const float a0 = a[i], b0 = b[i];
      a[i] = (_Float16)(a0 * p.cos - b0 * p.sin);
      b[i] = (_Float16)(b0 * p.cos + a0 * p.sin);
    }
  }
}

// The new tokens of one page: sequence, page of the sequence, slots.
struct Run {
  Sequence seq;
  int page, place, count;  // place of the first in the sequence
};

// Run number `wanted` (count 0: there are fewer).  One wave.
__device__ __forceinline__ Run find_run(const SeqArgs& s, int shift, int wanted) {
  int seen = 0;
  for (int b0 = 0; b0 < s.B; b0 += 64) {
    const Sequence q = sequence_at(s, shift, b0 + __lane_id());
    const int from = max(q.place0(), 0);
    const int runs = q.rows > 0 && q.length > 0 ? ((q.length - 1) >> shift) - (from >> shift) + 1 : 0;
    const int sum = seen + prefix_sum(runs);
    const unsigned long long owner = __ballot(sum > wanted && sum - runs <= wanted);
    if (owner != 0) {
      const int l = __builtin_ctzll(owner);
      Run r{pick(q, l), 0, 0, 0};
      const int first = __builtin_amdgcn_readlane(from, l);
      const int nth = wanted - (__builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(runs, l));
      r.page = (first >> shift) + nth;
      r.place = max(first, r.page << shift);
      r.count = min(r.seq.length, (r.page + 1) << shift) - r.place;
      return r;
    }
    seen = __builtin_amdgcn_readlane(sum, 63);
  }
  return Run{Sequence{0, 0, 0, 0}, 0, 0, 0};
}

__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a, CacheArgs c, SeqArgs s) {
  __shared__ Turn turns[kTokens][128];
  __shared__ half8_t least[2][128], most[2][128];
  const Run run = find_run(s, c.shift, blockIdx.x);
  if (run.count == 0) return;
  const int tid = threadIdx.x, D = c.dim, units = D / 16, pairs = a.rotary / 2;
  const bool keys = (int)blockIdx.y < c.heads;
  const int head0 = keys ? blockIdx.y : (blockIdx.y - c.heads) * kHeads;  // key head, or the first query head
  const int row0 = run.seq.row0 + run.place - run.seq.place0();
  const int number = s.tables[(int64_t)run.seq.index * s.width + run.page];
  const bool live = number >= 0 && number < c.pages;  // (no other page is written)
  const int slot0 = run.place & ((1 << c.shift) - 1);
  const int64_t tile = (((int64_t)(live ? number : 0) * c.heads + head0) << c.shift) + slot0;

  // keys: the first half of the threads; values: the second; or query heads
  const bool value = keys && tid >= kThreads / 2;
  const int mine = keys ? tid & (kThreads / 2 - 1) : tid;
  const int width = keys ? units : units * min(kHeads, a.q_heads - head0);  // units of a token
  const int lanes = (keys ? kThreads / 2 : kThreads) / width;               // tokens at a time
  const int u = mine % width, lane = mine / width;
  const int head = head0 + u / units;
  const bool turned = !value && 16 * (u % units) < a.rotary;
  const Unit unit = unit_of(u % units, value ? 0 : a.rotary, a.interleaved);
  const int64_t from = (int64_t)(keys ? a.q_heads + (value ? c.heads : 0) + head : head) * D;
  half8_t low[2], high[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    low[0][i] = low[1][i] = (_Float16)INFINITY;
    high[0][i] = high[1][i] = (_Float16)-INFINITY;
  }

  for (int t0 = 0; t0 < run.count; t0 += kTokens) {
    const int here = min(kTokens, run.count - t0);
    if (t0 > 0) __syncthreads();
    for (int i = tid; i < here * pairs; i += kThreads) {
      const int t = i / pairs, p = i - t * pairs;
      int position = run.place + t0 + t;
      if (a.positions) {
        const int axis = a.axis ? min(max(a.axis[p], 0), a.axes - 1) : 0;
        position = a.positions[(int64_t)(row0 + t0 + t) * a.axes + axis];
      }
      turns[t][p] = turn_of(position, a.inv_freq[p]);
    }
    __syncthreads();
    if (lane < lanes)
      for (int t = lane; t < here; t += lanes) {
        const int64_t row = row0 + t0 + t;
        const _Float16* x = a.x + row * a.ldx + from;
        half8_t lo = *reinterpret_cast<const half8_t*>(x + unit.lo), hi = *reinterpret_cast<const half8_t*>(x + unit.hi);
        if (turned) rotate(lo, hi, &turns[t][8 * (u % units)], a.interleaved);
        if (keys && !value) {
          low[0] = __builtin_elementwise_min(low[0], lo);
          low[1] = __builtin_elementwise_min(low[1], hi);
          high[0] = __builtin_elementwise_max(high[0], lo);
          high[1] = __builtin_elementwise_max(high[1], hi);
        }
        _Float16* to = keys ? (value ? c.v : c.k) + (tile + t0 + t) * D : a.q + row * a.ldq + (int64_t)head * D;
        if (!keys || live) {
          *reinterpret_cast<half8_t*>(to + unit.lo) = lo;
          *reinterpret_cast<half8_t*>(to + unit.hi) = hi;
        }
      }
  }

  if (!keys || !c.bounds || !live) return;  // (the same for the whole workgroup)
  if (!value) {
    least[0][mine] = low[0];
    least[1][mine] = low[1];
    most[0][mine] = high[0];
    most[1][mine] = high[1];
  }
  __syncthreads();
  if (tid >= units) return;
  for (int l = 1; l < lanes; ++l) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      low[i] = __builtin_elementwise_min(low[i], least[i][l * units + tid]);
      high[i] = __builtin_elementwise_max(high[i], most[i][l * units + tid]);
    }
  }
  _Float16* bounds = c.bounds + ((int64_t)number * c.heads + head0) * 2 * D;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    half8_t* at = reinterpret_cast<half8_t*>(bounds + (i ? unit.hi : unit.lo));
    half8_t* top = reinterpret_cast<half8_t*>(bounds + D + (i ? unit.hi : unit.lo));
    if (slot0 > 0) {
      low[i] = __builtin_elementwise_min(low[i], *at);
      high[i] = __builtin_elementwise_max(high[i], *top);
    }
    *at = low[i];
    *top = high[i];
  }
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, const CacheArgs& c, const SeqArgs& s, hipStream_t stream) {
  // pages with new tokens: one per token, or full ones and two more per sequence
  const int64_t runs = ((int64_t)s.T >> c.shift) + 2 * (int64_t)s.B;
  const dim3 grid((unsigned)(runs < s.T ? runs : s.T), c.heads + (a.q_heads + kHeads - 1) / kHeads);
  hipLaunchKernelGGL(append_kernel, grid, dim3(kThreads), 0, stream, a, c, s);
  return hipGetLastError();
}

}  // namespace awq
