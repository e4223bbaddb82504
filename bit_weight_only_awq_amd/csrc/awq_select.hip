// The pages that a token's queries attend to (awq_select_pages): per token and
// key head the `first` first pages, the `recent` last ones (the token's own
// among them) and, between those, the pages of the largest scores, in ascending
// order.
//
// Mathematics: with lo and hi a page's least and greatest key per channel, the
// largest product any key within them could have with query q is the sum over
// the channels of max(q lo, q hi), q hi where q > 0 and q lo where q < 0; a page's score is the sum of that over the key
// head's query heads.  Split by the sign of q it is Q+ . hi + Q- . lo, Q+ and Q-
// the sums of the heads' positive and negative parts: two multiply-adds per
// channel whatever the number of heads, in 64 bits, where the products of two
// halves are exact.  So a choice depends on the numbers, not on the order of the
// additions, and equal pages get equal scores (the lower page goes first).  A
// score that is not a number counts as the lowest.
//
// Bound: HBM, each page's bounds once, in the first kernel; the second finds the
// wanted number of largest scores by their bits, 8 at a time from the highest in
// which they differ, one workgroup per token and key head.
#include "awq_cache.hpp"

namespace awq {
namespace {

constexpr int kPages = 64;  // pages of a wave of the first kernel

// A score as a number whose unsigned order is the scores' order.
__device__ __forceinline__ uint64_t ordered(double v) {
  if (v != v) return 0;
  const uint64_t u = __builtin_bit_cast(uint64_t, v == 0.0 ? 0.0 : v);
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

__device__ __forceinline__ double swap_lanes(double v, int mask) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __shfl_xor((int)(uint32_t)u, mask), hi = __shfl_xor((int)(uint32_t)(u >> 32), mask);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// The pages that are scored: first .. have - recent - 1 of a row whose sequence has `have` pages up to its place.
struct Span {
  int place, have, from, to;
};
__device__ __forceinline__ Span span_of(const SelectArgs& a, const SeqArgs& s, int shift, int t, Sequence& q) {
  q = sequence_of(s, shift, t);
  const int place = q.rows ? t - q.row0 + q.place0() : -1;
  const int have = place < 0 ? 0 : (place >> shift) + 1;
  return Span{place, have, a.first, have > a.count ? have - a.recent : a.first};
}

// Scores of kPages pages of one token and key head: L lanes per row of bounds.
template <int D>
__global__ __launch_bounds__(256) void score_kernel(SelectArgs a, CacheArgs c, SeqArgs s, uint64_t* __restrict__ keys) {
  constexpr int CHUNKS = D / 4, L = CHUNKS <= 16 ? 16 : CHUNKS <= 32 ? 32 : 64, ROWS = 64 / L, STEPS = kPages / (16 * ROWS);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = blockIdx.x / c.heads, head = blockIdx.x % c.heads;
  Sequence q;
  const Span span = span_of(a, s, c.shift, t, q);
  const int p0 = span.from + (int)(blockIdx.y * 4 + wave) * kPages;
  if (p0 >= span.to) return;
  const int chunk = lane & (L - 1), row = lane / L;
  const bool high = chunk >= D / 8, live = chunk < CHUNKS;
  const int group = a.q_heads / c.heads, channel = 8 * (high ? chunk - D / 8 : chunk);
  double w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 0.0;
  if (live) {
    const _Float16* at = a.q + t * a.ldq + (int64_t)head * group * D + channel;
    for (int g = 0; g < group; ++g) {
      const half8_t v = *reinterpret_cast<const half8_t*>(at + (int64_t)g * D);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float f = v[i];
        w[i] += (double)(high ? (f > 0.0f ? f : f != f ? f : 0.0f) : (f < 0.0f ? f : 0.0f));
      }
    }
  }
  // channels that no head has on this side add 0, whatever the bound (infinities among them)
  u32x4 used;
#pragma unroll
  for (int i = 0; i < 4; ++i) used[i] = (w[2 * i] != 0.0 ? 0xFFFFu : 0u) | (w[2 * i + 1] != 0.0 ? 0xFFFF0000u : 0u);
  const int* table = s.tables + (int64_t)q.index * s.width;
  uint64_t* out = keys + ((int64_t)t * c.heads + head) * s.width;
#pragma unroll 1
  for (int step = 0; step < STEPS; ++step) {
    double sum[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int page = p0 + (step * 16 + j) * ROWS + row;
      u32x4 raw = u32x4(0u);
      if (live && page < span.to)
        raw = *reinterpret_cast<const u32x4*>(
            c.bounds + ((int64_t)page_number(c, table[page]) * c.heads + head) * 2 * D + 8 * chunk);
      const half8_t v = as_half8(raw & used);
      sum[j] = 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[j] = __builtin_fma(w[i], (double)(float)v[i], sum[j]);
    }
    // the lanes' sums: at each exchange half of the pages go to the other lane, then the rest of the lanes add up
#pragma unroll
    for (int h = 8; h >= 1; h >>= 1) {
      const bool upper = (lane & h) != 0;
#pragma unroll
      for (int j = 0; j < h; ++j) {
        const double keep = upper ? sum[j + h] : sum[j], give = upper ? sum[j] : sum[j + h];
        sum[j] = keep + swap_lanes(give, h);
      }
    }
    double total = sum[0];
#pragma unroll
    for (int m = 16; m < L; m <<= 1) total += swap_lanes(total, m);
    const int page = p0 + (step * 16 + (lane & 15)) * ROWS + row;
    if (chunk < 16 && page < span.to) out[page - span.from] = ordered(total);
  }
}

constexpr int kThreads = 1024;

__global__ __launch_bounds__(kThreads) void choose_kernel(SelectArgs a, CacheArgs c, SeqArgs s,
                                                          const uint64_t* __restrict__ keys) {
  __shared__ unsigned count[256];
  __shared__ unsigned part[kThreads / 64][2];
  __shared__ uint64_t bits[kThreads / 64];
  __shared__ unsigned found[2];
  const int t = blockIdx.x / c.heads, head = blockIdx.x % c.heads, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Sequence q;
  const Span span = span_of(a, s, c.shift, t, q);
  int* out = a.pages + ((int64_t)t * c.heads + head) * a.count;
  if (q.rows == 0) return;  // rows of no sequence stay as they are
  if (span.have <= a.count) {
    for (int i = tid; i < a.count; i += kThreads) out[i] = i < span.have ? i : -1;
    return;
  }
  const uint64_t* in = keys + ((int64_t)t * c.heads + head) * s.width;
  const int n = span.to - span.from;
  int wanted = a.count - a.first - a.recent;  // 0 <= wanted < n

  // the highest bit in which the scores differ
  uint64_t differ = 0;
  const uint64_t one = in[0];
  for (int i = tid; i < n; i += kThreads) differ |= in[i] ^ one;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint32_t lo = __shfl_xor((int)(uint32_t)differ, m), hi = __shfl_xor((int)(uint32_t)(differ >> 32), m);
    differ |= (uint64_t)hi << 32 | lo;
  }
  if (lane == 0) bits[wave] = differ;
  __syncthreads();
  differ = 0;
  for (int w = 0; w < kThreads / 64; ++w) differ |= bits[w];
  const int top = differ ? 64 - __builtin_clzll(differ) : 0;  // bits 0 .. top - 1 differ
  // the wanted-th largest: its bits from `top` down, 8 at a time
  uint64_t edge = top < 64 ? one >> top << top : 0;
  for (int shift = top; shift > 0 && wanted > 0;) {
    const int next = shift > 8 ? shift - 8 : 0, width = shift - next;
    for (int i = tid; i < 256; i += kThreads) count[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t k = in[i];
      if (shift == 64 || k >> shift == edge >> shift) atomicAdd(&count[(k >> next) & ((1u << width) - 1)], 1u);
    }
    __syncthreads();
    // the digit whose keys hold the wanted-th: lane l sums digits 255 - 4 l .. 252 - 4 l
    if (wave == 0) {
      unsigned c4[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += c4[i] = count[255 - 4 * lane - i];
      const unsigned upto = prefix_sum((int)sum);
      unsigned above = upto - sum;
      if (above < (unsigned)wanted && upto >= (unsigned)wanted) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (above < (unsigned)wanted && above + c4[i] >= (unsigned)wanted) {
            found[0] = 255 - 4 * lane - i;
            found[1] = above;
            break;
          }
          above += c4[i];
        }
      }
    }
    __syncthreads();
    edge |= (uint64_t)found[0] << next;
    wanted -= (int)found[1];
    shift = next;
    __syncthreads();
  }
  // in order: the pages above the edge, and the first `wanted` of those at it
  const bool none = a.count == a.first + a.recent;
  for (int i = tid; i < a.first; i += kThreads) out[i] = i;
  for (int i = tid; i < a.recent; i += kThreads) out[a.count - a.recent + i] = span.to + i;
  if (none) return;
  unsigned placed = a.first, ties = 0;
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + tid;
    const uint64_t k = i < n ? in[i] : 0;
    const bool tie = i < n && k == edge;
    const unsigned long long below = (1ull << lane) - 1, tied = __ballot(tie);
    if (lane == 0) part[wave][0] = __popcll(tied);
    __syncthreads();
    unsigned before = ties;
    for (int w = 0; w < kThreads / 64; ++w) {
      before += w < wave ? part[w][0] : 0;
      ties += part[w][0];
    }
    const bool take = i < n && (k > edge || (tie && before + __popcll(tied & below) < (unsigned)wanted));
    const unsigned long long taken = __ballot(take);
    if (lane == 0) part[wave][1] = __popcll(taken);
    __syncthreads();
    unsigned at = placed + __popcll(taken & below);
    for (int w = 0; w < kThreads / 64; ++w) {
      at += w < wave ? part[w][1] : 0;
      placed += part[w][1];
    }
    if (take) out[at] = span.from + i;
    __syncthreads();
  }
}

}  // namespace

size_t select_workspace_bytes(int T, int kv_heads, int width, int count) {
  return width > count ? ((size_t)T * kv_heads * width * 8 + 15) & ~(size_t)15 : 0;
}

hipError_t launch_select(const SelectArgs& a, const CacheArgs& c, const SeqArgs& s, void* workspace, hipStream_t stream) {
  uint64_t* keys = static_cast<uint64_t*>(workspace);
  if (s.width > a.count) {  // (otherwise no sequence has more pages than are wanted)
    const dim3 grid(s.T * c.heads, (s.width + 4 * kPages - 1) / (4 * kPages));
#define AWQ_SCORE(D) hipLaunchKernelGGL((score_kernel<D>), grid, dim3(256), 0, stream, a, c, s, keys)
    if (c.dim == 64) AWQ_SCORE(64);
    else if (c.dim == 96) AWQ_SCORE(96);
    else if (c.dim == 128) AWQ_SCORE(128);
    else AWQ_SCORE(256);
#undef AWQ_SCORE
  }
  hipLaunchKernelGGL(choose_kernel, dim3(s.T * c.heads), dim3(kThreads), 0, stream, a, c, s, keys);
  return hipGetLastError();
}

}  // namespace awq
