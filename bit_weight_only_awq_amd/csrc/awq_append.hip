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
// Bound: HBM for prompts (every row read and written once: 4.7 K tokens of 64 query
// and 8 key heads, 192 MB, in 43-45 us, 4.4 TB/s; a copy of as much takes 39); for a
// few tokens the launch and the chain lengths -> table -> row (1 token 4.4 us, 61
// 7.7).  One workgroup takes the new
// tokens of one page (so that nobody else writes its bounds) and one key head's
// keys and values, or kHeads query heads; the angles' sines and cosines are shared
// by the workgroup through LDS, one token of a thread at a time; the next token's
// row is under way meanwhile (without that 57 us; with two tokens at a time, in
// twice the registers, 46; held in 64 registers, which spills, 57).
#include "awq_cache.hpp"

namespace awq {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;    // query heads of a workgroup
constexpr int kTurns = kThreads / 2 * 8;  // of the tokens that a workgroup has at a time

struct Turn {
  float cos, sin;
};

__device__ __forceinline__ Turn turn_of(double t) {  // (an angle in quarter turns)
  const double whole = __builtin_rint(t);
  const float x = (float)(t - whole) * 1.5707963267948966f, y = x * x;
  const float sin = x + x * y * (-1.6666666666666666e-1f + y * (8.3333333333333333e-3f + y * (-1.984126984126984e-4f +
                                                                                            y * 2.7557319223985893e-6f)));
  const float cos = 1.0f + y * (-0.5f + y * (4.1666666666666664e-2f + y * (-1.3888888888888889e-3f +
                                                                          y * 2.48015873015873e-5f)));
  const int quarter = (int)(whole - 4.0 * __builtin_rint(whole * 0.25)) & 3;
  const float s = quarter & 1 ? cos : sin, c = quarter & 1 ? sin : cos;
  return Turn{quarter == 1 || quarter == 2 ? -c : c, quarter >= 2 ? -s : s};
}

// Sixteen channels of a head: two chunks of eight, half of the rotated part (or
// of the rest) apart, so that neighbouring threads have neighbouring chunks.  A
// unit of the rotated part holds the pairs of both: 8 u .. 8 u + 7, or, where
// pairs are neighbours, four of each half.
struct Unit {
  int lo, hi;
};
__device__ __forceinline__ Unit unit_of(int u, int rotary, int dim) {
  const int lo = 8 * u;
  return 2 * lo < rotary ? Unit{lo, rotary / 2 + lo} : Unit{rotary / 2 + lo, dim / 2 + lo};
}
// Where a token's pair p is among its turns: quarters of units side by side (a
// thread reads its four with its neighbours'; four conflict cycles per access are
// counted, writing the turns among them).
__device__ __forceinline__ int place_of(int p, int rotary, bool interleaved) {
  const int units = rotary / 16, far = interleaved && p >= rotary / 4, q = p - (far ? rotary / 4 : 0);
  const int u = interleaved ? q / 4 : q / 8, quarter = interleaved ? 2 * far + q % 4 / 2 : q % 8 / 2;
  return 2 * (quarter * units + u) + (p & 1);
}

__device__ __forceinline__ void rotate(half8_t& a, half8_t& b, const Turn* turn, bool interleaved) {
  half8_t p = a, q = b;
  if (interleaved) {
    p = __builtin_shufflevector(a, b, 0, 2, 4, 6, 8, 10, 12, 14);
    q = __builtin_shufflevector(a, b, 1, 3, 5, 7, 9, 11, 13, 15);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float p0 = p[i], q0 = q[i];
    p[i] = (_Float16)(p0 * turn[i].cos - q0 * turn[i].sin);
    q[i] = (_Float16)(q0 * turn[i].cos + p0 * turn[i].sin);
  }
  a = p;
  b = q;
  if (interleaved) {
    a = __builtin_shufflevector(p, q, 0, 8, 1, 9, 2, 10, 3, 11);
    b = __builtin_shufflevector(p, q, 4, 12, 5, 13, 6, 14, 7, 15);
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
  __shared__ float4_t turns[kTurns / 2];
  __shared__ half8_t least[2][128], most[2][128];
  const int tid = threadIdx.x, D = c.dim, units = D / 16, pairs = a.rotary / 2;
  // the thread's pair of the sines and its first token
  const int pair = pairs > 0 ? tid % pairs : 0, tokens = pairs > 0 ? kThreads / pairs : 0;
  const int token = pairs > 0 ? tid / pairs : 0, at = place_of(pair, a.rotary, a.interleaved);
  const double freq = pairs > 0 ? (double)a.inv_freq[pair] * 0.63661977236758134 : 0.0;  // in quarter turns: 2 / pi
  const int axis = a.axis && pairs > 0 ? min(max(a.axis[pair], 0), a.axes - 1) : 0;
  const Run run = find_run(s, c.shift, blockIdx.x);
  if (run.count == 0) return;
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
  const int width = keys ? units : units * kHeads;           // units of a token
  const int lanes = (keys ? kThreads / 2 : kThreads) / width;  // tokens at a time
  const int u = mine % width, lane = mine / width;
  const int head = head0 + u / units;
  const bool has = lane < lanes && (keys || head < a.q_heads);
  const bool turned = !value && 16 * (u % units) < a.rotary;
  const Unit unit = unit_of(u % units, value ? 0 : a.rotary, D);
  const _Float16* x = a.x + row0 * a.ldx + (int64_t)(keys ? a.q_heads + (value ? c.heads : 0) + head : head) * D;
  _Float16* to = keys ? (value ? c.v : c.k) + tile * D : a.q + row0 * a.ldq + (int64_t)head * D;
  const int64_t ldto = keys ? D : a.ldq;
  half8_t low[2], high[2], lo, hi;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    low[0][i] = low[1][i] = (_Float16)INFINITY;
    high[0][i] = high[1][i] = (_Float16)-INFINITY;
  }
  const auto load = [&](int t) {
    if (has && t < run.count) {
      lo = *reinterpret_cast<const half8_t*>(x + t * a.ldx + unit.lo);
      hi = *reinterpret_cast<const half8_t*>(x + t * a.ldx + unit.hi);
    }
  };

  load(lane);
  for (int t0 = 0; t0 < run.count; t0 += lanes) {
    const int here = min(lanes, run.count - t0), t = t0 + lane;
    if (t0 > 0) __syncthreads();
    if (token < tokens)
      for (int i = token; i < here; i += tokens) {
        const int position = a.positions ? a.positions[(int64_t)(row0 + t0 + i) * a.axes + axis] : run.place + t0 + i;
        reinterpret_cast<Turn*>(turns)[i * pairs + at] = turn_of(position * freq);
      }
    __syncthreads();
    half8_t first = lo, second = hi;
    load(t + lanes);
    if (!has || lane >= here) continue;
    if (turned) {
      Turn turn[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4_t two = turns[lane * (pairs / 2) + k * (a.rotary / 16) + u % units];
        turn[2 * k] = Turn{two[0], two[1]};
        turn[2 * k + 1] = Turn{two[2], two[3]};
      }
      rotate(first, second, turn, a.interleaved);
    }
    if (keys && !value) {
      low[0] = __builtin_elementwise_min(low[0], first);
      low[1] = __builtin_elementwise_min(low[1], second);
      high[0] = __builtin_elementwise_max(high[0], first);
      high[1] = __builtin_elementwise_max(high[1], second);
    }
    if (!keys || live) {
      *reinterpret_cast<half8_t*>(to + t * ldto + unit.lo) = first;
      *reinterpret_cast<half8_t*>(to + t * ldto + unit.hi) = second;
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
