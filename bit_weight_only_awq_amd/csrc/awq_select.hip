// The pages that a token's queries attend to (awq_select_pages): per token and
// key head the `first` first pages, the `recent` last ones (the token's own
// among them) and, between those, the pages of the largest scores, in ascending
// order.
//
// Mathematics: with lo and hi a page's least and greatest key per channel, the
// largest product any key within them could have with query q is the sum over
// the channels of max(q lo, q hi), q hi where q > 0 and q lo where q < 0; a page's
// score is the sum of that over the key head's query heads.  Split by the sign of q it is Q+ . hi + Q- . lo, Q+ and Q-
// the sums of the heads' positive and negative parts: two multiply-adds per
// channel whatever the number of heads, in 64 bits, where a sum is rounded only if it
// takes more than 53 of them.  Every page's sums are made in the same order, so equal
// pages get equal scores (the lower page goes first).  A score that is not a number
// counts as the lowest.
//
// Bound: HBM, each page's bounds once, in the first kernel (32 tokens of up to 1024
// pages, 95 MB: 26 us, 3.7 TB/s, 10 of them fp64 instructions; 1 token of 6251
// pages, 26 MB: 9.6-10.8); the second finds the wanted number of largest scores by their
// bits, 8 at a time from the highest in which they differ, one workgroup per token and
// key head: a chain of reads and rounds (8.5 us in both cases).  Narrow tables take
// both steps in one launch.
#include "awq_cache.hpp"

namespace awq {
namespace {

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

// At each exchange half of a lane's sums go to the lane H away, which has its share of them, and as many come back.
template <int H>
__device__ __forceinline__ void halve(double (&sum)[16], int lane) {
  const bool upper = (lane & H) != 0;
#pragma unroll
  for (int j = 0; j < H; ++j) {
    const double keep = upper ? sum[j + H] : sum[j], give = upper ? sum[j] : sum[j + H];
    sum[j] = keep + swap_lanes(give, H);
  }
  if constexpr (H > 1) halve<H / 2>(sum, lane);
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

// Scores of 16 ROWS pages of one token and key head per wave: L lanes per row of bounds.
template <int D>
struct Score {
  static constexpr int CHUNKS = D / 4, L = CHUNKS <= 16 ? 16 : CHUNKS <= 32 ? 32 : 64, ROWS = 64 / L, PAGES = 16 * ROWS;
};

// Scores of pages p0 .. p0 + PAGES - 1, then of those `step` further, below p1, by one wave, of token t and a key head:
// put(page - span.from, score).
template <int D, typename Put>
__device__ __forceinline__ void score_pages(const SelectArgs& a, const CacheArgs& c, const SeqArgs& s, const Sequence& q,
                                            int t, int head, int p0, int step, int p1, int from, Put put) {
  using P = Score<D>;
  constexpr int L = P::L;
  const int lane = threadIdx.x & 63, chunk = lane & (L - 1), row = lane / L;
  const bool high = chunk >= D / 8, live = chunk < P::CHUNKS;
  const int group = a.q_heads / c.heads, channel = 8 * (high ? chunk - D / 8 : chunk);
  // the pages' numbers, one per lane, while the queries arrive
  const int* table = s.tables + (int64_t)q.index * s.width;
  auto number_of = [&](int at) { return page_number(c, table[min(at + min(lane, P::PAGES - 1), p1 - 1)]); };
  int number = number_of(p0);
  double w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 0.0;
  {
    const _Float16* at = a.q + t * a.ldq + (int64_t)head * group * D + (live ? channel : 0);
    for (int g0 = 0; g0 < group; g0 += 4) {
      half8_t v[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) v[g] = *reinterpret_cast<const half8_t*>(at + (int64_t)min(g0 + g, group - 1) * D);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        // (the sign picks the side: halves with the other sign become 0)
        const uint32_t mine = high ? 0xFFFFFFFFu : 0u, in = live && g0 + g < group ? 0xFFFFFFFFu : 0u;
        const u32x4 bits = __builtin_bit_cast(u32x4, v[g]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t pair = bits[i];
          const uint32_t negative = ((int)pair < 0 ? 0xFFFF0000u : 0u) | (pair & 0x8000u ? 0xFFFFu : 0u);
          const half2_t side = as_half2(pair & (negative ^ mine) & in);
          w[2 * i] += (double)(float)side[0];
          w[2 * i + 1] += (double)(float)side[1];
        }
      }
    }
  }
  // channels that no head has on this side add 0, whatever the bound (infinities among them)
  u32x4 used;
#pragma unroll
  for (int i = 0; i < 4; ++i) used[i] = (w[2 * i] != 0.0 ? 0xFFFFu : 0u) | (w[2 * i + 1] != 0.0 ? 0xFFFF0000u : 0u);
#pragma unroll 1
  for (; p0 < p1; p0 += step) {
    u32x4 raw[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int64_t page = __shfl(number, j * P::ROWS + row);
      raw[j] = *reinterpret_cast<const u32x4*>(c.bounds + (page * c.heads + head) * 2 * D + (live ? 8 * chunk : 0));
    }
    if (p0 + step < p1) number = number_of(p0 + step);
    double sum[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const half8_t v = as_half8(raw[j] & used);
      sum[j] = 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[j] = __builtin_fma(w[i], (double)(float)v[i], sum[j]);
    }
    // the lanes' sums, page by page, then those of the lanes 16 and 32 away
    halve<8>(sum, lane);
    double total = sum[0];
#pragma unroll
    for (int m = 16; m < L; m <<= 1) total += swap_lanes(total, m);
    const int page = p0 + (lane & 15) * P::ROWS + row;
    if (chunk < 16 && page < p1) put(page - from, ordered(total));
  }
}

template <int D>
__global__ __launch_bounds__(256) void score_kernel(SelectArgs a, CacheArgs c, SeqArgs s, int batches,
                                                    uint64_t* __restrict__ keys) {
  constexpr int PAGES = Score<D>::PAGES;
  const int wave = threadIdx.x >> 6, t = blockIdx.x / c.heads, head = blockIdx.x % c.heads;
  Sequence q;
  const Span span = span_of(a, s, c.shift, t, q);
  const int p0 = span.from + (int)(blockIdx.y * 4 + wave) * batches * PAGES;
  if (p0 >= span.to) return;
  uint64_t* out = keys + ((int64_t)t * c.heads + head) * s.width;
  score_pages<D>(a, c, s, q, t, head, p0, PAGES, min(span.to, p0 + batches * PAGES), span.from,
                 [&](int i, uint64_t score) { out[i] = score; });
}

constexpr int kScoreWaves = 4096;  // four per SIMD

constexpr int kKept = 8;  // scores that a thread holds at a time: of 1024 threads numbers tid, tid + 1024, ... of 8192

// The place of each flagged score among all flagged ones before it, `placed` so far.
struct Places {
  unsigned at[kKept];
};
template <int WAVES>
__device__ __forceinline__ Places places_of(const bool (&flag)[kKept], unsigned* part, unsigned& placed) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Places p;
#pragma unroll
  for (int k = 0; k < kKept; ++k) {
    const unsigned long long all = __ballot(flag[k]);
    p.at[k] = __popcll(all & ((1ull << lane) - 1));
    if (lane == 0) part[k * WAVES + wave] = __popcll(all);
  }
  __syncthreads();
  constexpr int COUNTS = kKept * WAVES, EACH = COUNTS / 64;
  static_assert(EACH == 1 || EACH == 2, "one or two counts per lane");
  if (wave == 0) {
    const unsigned x = part[EACH * lane], y = EACH == 2 ? part[EACH * lane + 1] : 0, upto = prefix_sum((int)(x + y));
    part[EACH * lane] = upto - x - y;
    if (EACH == 2) part[EACH * lane + 1] = upto - y;
    if (lane == 63) part[COUNTS] = upto;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kKept; ++k) p.at[k] += placed + part[k * WAVES + wave];
  placed += part[COUNTS];
  __syncthreads();
  return p;
}

// The pages of a token and key head that are chosen whatever the scores; whether that is all.
template <int THREADS>
__device__ __forceinline__ bool choose_fixed(const SelectArgs& a, const Span& span, int* out) {
  const int tid = threadIdx.x;
  if (span.have <= a.count) {
    for (int i = tid; i < a.count; i += THREADS) out[i] = i < span.have ? i : -1;
    return true;
  }
  for (int i = tid; i < a.first; i += THREADS) out[i] = i;
  for (int i = tid; i < a.recent; i += THREADS) out[a.count - a.recent + i] = span.to + i;
  return a.count == a.first + a.recent;
}

// Of scores in[0 .. span.to - span.from - 1] the largest, by a workgroup.
template <int THREADS>
__device__ __forceinline__ void choose(const SelectArgs& a, const Span& span, int* out, const uint64_t* in) {
  constexpr int WAVES = THREADS / 64;
  __shared__ unsigned count[256], part[kKept * WAVES + 1], found[3];
  __shared__ uint64_t bits[WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = span.to - span.from, rounds = (n + kKept * THREADS - 1) / (kKept * THREADS);
  int wanted = a.count - a.first - a.recent;  // 0 < wanted < n

  uint64_t kept[kKept];
  auto read = [&](int round) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
      const int i = (round * kKept + k) * THREADS + tid;
      kept[k] = i < n ? in[i] : 0;
    }
  };
  auto number = [&](int round, int k) __attribute__((always_inline)) { return (round * kKept + k) * THREADS + tid; };

  // the highest bit in which the scores differ
  const uint64_t one = in[0];
  uint64_t differ = 0;
  for (int r = 0; r < rounds; ++r) {
    read(r);
#pragma unroll
    for (int k = 0; k < kKept; ++k) differ |= number(r, k) < n ? kept[k] ^ one : 0;
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint32_t lo = __shfl_xor((int)(uint32_t)differ, m), hi = __shfl_xor((int)(uint32_t)(differ >> 32), m);
    differ |= (uint64_t)hi << 32 | lo;
  }
  if (lane == 0) bits[wave] = differ;
  if (tid < 256) count[tid] = 0;
  __syncthreads();
  differ = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) differ |= bits[w];
  const int top = differ ? 64 - __builtin_clzll(differ) : 0;  // bits 0 .. top - 1 differ
  // the wanted-th largest: its bits from `top` down, 8 at a time, until no more scores share those found than are
  // wanted of them
  uint64_t edge = top < 64 ? one >> top << top : 0;
  bool ties = true;
  for (int shift = top; shift > 0 && ties;) {
    const int next = shift > 8 ? shift - 8 : 0;
    for (int r = 0; r < rounds; ++r) {
      if (rounds > 1) read(r);
#pragma unroll
      for (int k = 0; k < kKept; ++k)
        if (number(r, k) < n && (shift == 64 || kept[k] >> shift == edge >> shift))
          atomicAdd(&count[(kept[k] >> next) & 255 & ((1u << (shift - next)) - 1)], 1u);
    }
    __syncthreads();
    // the digit whose scores hold the wanted-th: lane l sums digits 255 - 4 l .. 252 - 4 l
    if (wave == 0) {
      unsigned c4[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += c4[i] = count[255 - 4 * lane - i];
      const unsigned upto = prefix_sum((int)sum);
      unsigned above = upto - sum;
      bool done = above >= (unsigned)wanted || upto < (unsigned)wanted;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!done && above + c4[i] >= (unsigned)wanted) {
          found[0] = 255 - 4 * lane - i;
          found[1] = above;
          found[2] = c4[i];
          done = true;
        }
        above += c4[i];
      }
    }
    __syncthreads();
    edge |= (uint64_t)found[0] << next;
    wanted -= (int)found[1];
    ties = found[2] != (unsigned)wanted;
    shift = next;
    if (tid < 256) count[tid] = 0;
    __syncthreads();
  }
  // in order: the pages at or above the edge; with ties, those above it and the first `wanted` of those at it
  unsigned placed = a.first, tied = 0;
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) read(r);
    bool take[kKept];
    if (ties) {
      bool equal[kKept];
#pragma unroll
      for (int k = 0; k < kKept; ++k) equal[k] = number(r, k) < n && kept[k] == edge;
      const Places p = places_of<WAVES>(equal, part, tied);
#pragma unroll
      for (int k = 0; k < kKept; ++k)
        take[k] = number(r, k) < n && (kept[k] > edge || (equal[k] && p.at[k] < (unsigned)wanted));
    } else {
#pragma unroll
      for (int k = 0; k < kKept; ++k) take[k] = number(r, k) < n && kept[k] >= edge;
    }
    const Places p = places_of<WAVES>(take, part, placed);
#pragma unroll
    for (int k = 0; k < kKept; ++k)
      if (take[k]) out[p.at[k]] = span.from + number(r, k);
  }
}

__global__ __launch_bounds__(1024) void choose_kernel(SelectArgs a, CacheArgs c, SeqArgs s, const uint64_t* __restrict__ keys) {
  const int t = blockIdx.x / c.heads, head = blockIdx.x % c.heads;
  Sequence q;
  const Span span = span_of(a, s, c.shift, t, q);
  int* out = a.pages + ((int64_t)t * c.heads + head) * a.count;
  if (q.rows == 0) return;  // rows of no sequence stay as they are
  if (choose_fixed<1024>(a, span, out)) return;
  choose<1024>(a, span, out, keys + ((int64_t)t * c.heads + head) * s.width);
}

// Both in one launch, the scores in LDS, where the tables are so narrow that one workgroup reads a row's bounds in the
// time of a launch (17 tokens of 30 key heads, 24 pages: select and attend 66.6 us, in two launches 76; 1 token of 8 pages of
// 128 channels 31.3, 36; but 13 tokens of one head, 950 pages of 256 channels 50.5, 37.5).
constexpr int kAlone = 512;  // pages

template <int D>
__global__ __launch_bounds__(512) void select_kernel(SelectArgs a, CacheArgs c, SeqArgs s) {
  __shared__ uint64_t keys[kAlone];
  const int t = blockIdx.x / c.heads, head = blockIdx.x % c.heads;
  Sequence q;
  const Span span = span_of(a, s, c.shift, t, q);
  int* out = a.pages + ((int64_t)t * c.heads + head) * a.count;
  if (q.rows == 0) return;
  if (choose_fixed<512>(a, span, out)) return;  // (the same for the whole workgroup)
  constexpr int PAGES = Score<D>::PAGES;
  const int p0 = span.from + (int)(threadIdx.x >> 6) * PAGES;
  if (p0 < span.to)
    score_pages<D>(a, c, s, q, t, head, p0, 8 * PAGES, span.to, span.from, [&](int i, uint64_t score) { keys[i] = score; });
  __syncthreads();
  choose<512>(a, span, out, keys);
}

template <int D>
void launch_score(const SelectArgs& a, const CacheArgs& c, const SeqArgs& s, uint64_t* keys, hipStream_t stream) {
  constexpr int PAGES = Score<D>::PAGES;
  // a wave's pages: one batch where that fills the chip, more where the queries' sums would be formed too often
  const int64_t all = (int64_t)s.T * c.heads * ((s.width + PAGES - 1) / PAGES), want = all / kScoreWaves;
  int batches = want < 1 ? 1 : want > 8 ? 8 : (int)want;
  constexpr int kMostGroups = 65535;  // (of a launch in y)
  batches = max(batches, s.width / (4 * PAGES) / kMostGroups + 1);
  const int pages = 4 * batches * PAGES;
  hipLaunchKernelGGL((score_kernel<D>), dim3(s.T * c.heads, (s.width + pages - 1) / pages), dim3(256), 0, stream, a, c, s,
                     batches, keys);
}

}  // namespace

size_t select_workspace_bytes(int T, int kv_heads, int width, int count) {
  return width > count && width > kAlone ? ((size_t)T * kv_heads * width * 8 + 15) & ~(size_t)15 : 0;
}

hipError_t launch_select(const SelectArgs& a, const CacheArgs& c, const SeqArgs& s, void* workspace, hipStream_t stream) {
  uint64_t* keys = static_cast<uint64_t*>(workspace);
#define AWQ_SELECT(D)                                                                                       \
  if (s.width <= kAlone) hipLaunchKernelGGL((select_kernel<D>), dim3(s.T * c.heads), dim3(512), 0, stream, a, c, s); \
  else if (s.width > a.count) launch_score<D>(a, c, s, keys, stream)
  if (c.dim == 64) { AWQ_SELECT(64); }
  else if (c.dim == 96) { AWQ_SELECT(96); }
  else if (c.dim == 128) { AWQ_SELECT(128); }
  else { AWQ_SELECT(256); }
#undef AWQ_SELECT
  if (s.width > kAlone)  // (with no more pages than are wanted there are no scores, and none are looked at)
    hipLaunchKernelGGL(choose_kernel, dim3(s.T * c.heads), dim3(1024), 0, stream, a, c, s, keys);
  return hipGetLastError();
}

}  // namespace awq
