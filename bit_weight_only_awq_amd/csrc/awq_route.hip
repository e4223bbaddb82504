// The expert router (awq_route_experts): for each token the top_k largest of
// its E logits (the lower index first among equal ones), their softmax
// weights, and the slots (token t's j-th choice is slot t * top_k + j) sorted
// by expert.
//
// Mathematics: with m the token's largest logit, w_j = exp(l_j - m) / S, S the
// sum of exp(l - m) over the chosen logits (renormalize) or over all of them,
// in fp32.  A logit of -inf or NaN is never chosen: its slot has id -1,
// weight 0 and position -1.  With m = +inf the +inf logits share the weight.
//
// Bound: latency for a few tokens (one launch, 3-6 us), the vector instructions of
// the picks for many: 126 per pick of a wave with 8 logits per lane (the owning
// lane searches its logits and takes their maximum again, and the others wait).  LG
// lanes hold a token's logits, consecutive ones per lane, so the lowest lane with
// the maximum also has the lowest index; a maximum over the lanes is log2(LG)
// register exchanges (DPP).
//
// The sort is a counting sort without atomics on anything but bits and integer
// sums: a token chooses an expert at most once, so the choices of a block's 64
// tokens for one expert are one 64-bit word, and a slot's rank among its
// expert's slots is a population count.  Up to 64 tokens one launch does it
// all; more blocks write their counts (a byte per expert) and a second launch adds up
// the counts of the blocks before each; past 512 blocks a launch between the two
// sums the counts along the blocks, so that the work stays linear.
//
// Measured (us): 1 token of 8 experts, top 2: 2.6; 64 tokens: 2.9; 1024 of 64, top
// 6: 10.3; 16384 of 128, top 8: 18.3 (choosing 12, placing 7), and 51.5 with 256
// tokens per block.
#include "awq_epilogue.hpp"
#include "awq_launch_fused.hpp"

namespace awq {
namespace {

constexpr int kTokens = 64;       // tokens per block: the bits of a mask
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;
constexpr int kSumBlocks = 512;   // blocks whose counts every block adds up for itself

// Largest of v (sum of v) over groups of LG consecutive lanes, in every lane.
template <int LG, typename Op>
__device__ __forceinline__ float group_reduce(float v, Op op) {
  v = op(v, row_rotate<0x141>(v));                        // row_half_mirror
  v = op(v, row_rotate<0x4E>(v));                         // quad_perm [2, 3, 0, 1]
  v = op(v, row_rotate<0xB1>(v));                         // quad_perm [1, 0, 3, 2]
  if constexpr (LG >= 16) v = op(v, row_rotate<0x128>(v));  // row_ror:8
  if constexpr (LG >= 32) v = op(v, __shfl_xor(v, 16));
  if constexpr (LG >= 64) v = op(v, __shfl_xor(v, 32));
  return v;
}
template <int LG>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<LG>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int LG>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<LG>(v, [](float a, float b) { return a + b; });
}

__device__ __forceinline__ float exp_below(float l, float m) { return l == m ? 1.0f : expf(l - m); }

// What a block keeps of its tokens' choices.
struct Choices {
  unsigned long long mask[kMaxExperts];  // bit t: the block's token t chose the expert
  int id[kTokens * kMaxTopK];
  float share[kTokens * kMaxTopK];       // exp(l - m)
};

// The block's tokens' choices: LG lanes per token, EPL consecutive logits per lane.
template <int LG, int EPL, typename T>
__device__ __forceinline__ void choose(const T* __restrict__ logits, int64_t ld, int tokens, int E, int top_k,
                                       bool renormalize, int* __restrict__ ids, float* __restrict__ weights,
                                       Choices& c) {
  const int lane = threadIdx.x & 63, l = lane & (LG - 1), base = lane & ~(LG - 1);
  const int per_pass = blockDim.x / LG;
  for (int t0 = 0; t0 < tokens; t0 += per_pass) {
    const int t = t0 + threadIdx.x / LG;
    const bool live = t < tokens;
    float v[EPL], mine = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = l * EPL + i;
      v[i] = live && e < E ? (float)logits[t * ld + e] : -INFINITY;
      if (v[i] != v[i]) v[i] = -INFINITY;
      mine = fmaxf(mine, v[i]);
    }
    const float m = group_max<LG>(mine);
    float all = 0.0f;
    if (!renormalize) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) all += v[i] == -INFINITY ? 0.0f : exp_below(v[i], m);
      all = group_sum<LG>(all);
    }
    float best = m, sum = 0.0f;
    for (int j = 0; j < top_k; ++j) {
      const bool any = best != -INFINITY;
      const float share = any ? exp_below(best, m) : 0.0f;
      sum += share;
      const int owner = __builtin_ctzll(__ballot(mine == best) >> base);
      if (l == owner && live) {
        int at = -1;
        if (any) {
          // the first of the lane's logits that equals it, taken out
          mine = -INFINITY;
#pragma unroll
          for (int i = 0; i < EPL; ++i) {
            if (at < 0 && v[i] == best) {
              at = l * EPL + i;
              v[i] = -INFINITY;
            }
            mine = fmaxf(mine, v[i]);
          }
          atomicOr(&c.mask[at], 1ull << t);
        }
        c.id[t * top_k + j] = at;
        c.share[t * top_k + j] = share;
      }
      best = group_max<LG>(mine);
    }
    // (written and read within one wave, in order)
    const float total = renormalize ? sum : all;
    if (live)
      for (int j = l; j < top_k; j += LG) {
        const int s = t * top_k + j;
        ids[s] = c.id[s];
        weights[s] = total > 0.0f ? c.share[s] / total : 0.0f;
      }
  }
}

// start[e] (LDS) holds expert e's slots in all blocks: replaced by the sum over
// the experts below; start[E] the total.  One wave.
__device__ __forceinline__ void scan_experts(int* start, int E) {
  if (threadIdx.x < 64) {
    int seen = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + threadIdx.x;
      const int n = e < E ? start[e] : 0;
      const int sum = prefix_sum(n);
      if (e < E) start[e] = seen + sum - n;
      seen += __builtin_amdgcn_readlane(sum, 63);
    }
    if (threadIdx.x == 0) start[E] = seen;
  }
  __syncthreads();
}

// Positions and rows of the block's slots, from the masks and the place of
// the block's first slot of each expert.
__device__ __forceinline__ void place(const int* id, int t0, int tokens, int top_k, const unsigned long long* mask,
                                      const int* first, int* __restrict__ positions, int* __restrict__ rows) {
  for (int s = threadIdx.x; s < tokens * top_k; s += blockDim.x) {
    const int e = id[s], t = s / top_k;
    int at = -1;
    if (e >= 0) {
      at = first[e] + __popcll(mask[e] & ((1ull << t) - 1));
      rows[at] = t0 * top_k + s;
    }
    positions[(int64_t)t0 * top_k + s] = at;
  }
}

// One block: the choices of kTokens tokens, and either the whole sort (one
// block in the grid) or the block's counts per expert, a byte each.
template <int LG, int EPL, typename T>
__global__ __launch_bounds__(1024) void route_kernel(const T* __restrict__ logits, int ld, int tokens, int E, int top_k,
                                                     int renormalize, int* __restrict__ ids,
                                                     float* __restrict__ weights, int* __restrict__ offsets,
                                                     int* __restrict__ rows, int* __restrict__ positions,
                                                     uint8_t* __restrict__ counts) {
  __shared__ Choices c;
  __shared__ int start[kMaxExperts + 1];
  const int t0 = blockIdx.x * kTokens, here = min(kTokens, tokens - t0);
  for (int e = threadIdx.x; e < E; e += blockDim.x) c.mask[e] = 0;
  __syncthreads();
  choose<LG, EPL, T>(logits + (int64_t)t0 * ld, ld, here, E, top_k, renormalize != 0, ids + (int64_t)t0 * top_k,
                     weights + (int64_t)t0 * top_k, c);
  __syncthreads();
  if (gridDim.x > 1) {
    const int pitch = (E + 3) & ~3;
    for (int e = threadIdx.x; e < pitch; e += blockDim.x)
      counts[(int64_t)blockIdx.x * pitch + e] = e < E ? (uint8_t)__popcll(c.mask[e]) : 0;
    return;
  }
  for (int e = threadIdx.x; e < E; e += blockDim.x) start[e] = __popcll(c.mask[e]);
  __syncthreads();
  scan_experts(start, E);
  for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = start[e];
  place(c.id, 0, here, top_k, c.mask, start, positions, rows);
  for (int i = start[E] + threadIdx.x; i < tokens * top_k; i += blockDim.x) rows[i] = -1;
}

// Sums along the blocks for 4 experts: base[b][e] = the slots of expert e in the
// blocks before b, base[blocks][e] in all.
__global__ __launch_bounds__(1024) void route_sum_kernel(const uint32_t* __restrict__ counts, int blocks, int words,
                                                         int* __restrict__ base) {
  __shared__ int part[16][4];
  const int w = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = (blocks + 1023) / 1024, b0 = threadIdx.x * per, b1 = min(blocks, b0 + per);
  int sum[4] = {0, 0, 0, 0}, first[4];
  for (int b = b0; b < b1; ++b) {
    const uint32_t v = counts[(int64_t)b * words + w];
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] += (v >> (8 * i)) & 255u;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int upto = prefix_sum(sum[i]);
    first[i] = upto - sum[i];
    if (lane == 63) part[wave][i] = upto;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i)
    for (int v = 0; v < wave; ++v) first[i] += part[v][i];
  for (int b = b0; b < b1; ++b) {
    const uint32_t v = counts[(int64_t)b * words + w];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      base[((int64_t)b * words + w) * 4 + i] = first[i];
      first[i] += (v >> (8 * i)) & 255u;
    }
  }
  if (threadIdx.x == 1023)
#pragma unroll
    for (int i = 0; i < 4; ++i) base[((int64_t)blocks * words + w) * 4 + i] = first[i];
}

// Offsets, and the positions and rows of one block's slots; `base` from
// route_sum_kernel, or NULL: the block adds up the counts itself.
__global__ __launch_bounds__(1024) void route_place_kernel(const int* __restrict__ ids, int tokens, int E, int top_k,
                                                           const uint32_t* __restrict__ counts,
                                                           const int* __restrict__ base, int* __restrict__ offsets,
                                                           int* __restrict__ rows, int* __restrict__ positions) {
  __shared__ unsigned long long mask[kMaxExperts];
  __shared__ int start[kMaxExperts + 1], before[kMaxExperts], id[kTokens * kMaxTopK];
  const int b = blockIdx.x, blocks = gridDim.x, t0 = b * kTokens, here = min(kTokens, tokens - t0);
  const int words = (E + 3) >> 2;
  for (int e = threadIdx.x; e < 4 * words; e += blockDim.x) {
    mask[e] = 0;
    before[e] = base ? base[(int64_t)b * words * 4 + e] : 0;
    start[e] = base ? base[(int64_t)blocks * words * 4 + e] : 0;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < here * top_k; s += blockDim.x) {
    const int e = ids[(int64_t)t0 * top_k + s];
    id[s] = e;
    if (e >= 0) atomicOr(&mask[e], 1ull << (s / top_k));
  }
  if (!base) {
    // four experts per word, two 16-bit sums per register (at most 512 blocks of 64)
    const int sets = blockDim.x / words, w = threadIdx.x % words, set = threadIdx.x / words;
    if (set < sets) {
      uint32_t lo = 0, hi = 0, lo_before = 0, hi_before = 0;
#pragma unroll 4
      for (int r = set; r < blocks; r += sets) {
        const uint32_t v = counts[(int64_t)r * words + w], even = v & 0x00FF00FFu, odd = (v >> 8) & 0x00FF00FFu;
        lo += even;
        hi += odd;
        lo_before += r < b ? even : 0u;
        hi_before += r < b ? odd : 0u;
      }
      atomicAdd(&start[4 * w], (int)(lo & 0xFFFFu));
      atomicAdd(&start[4 * w + 1], (int)(hi & 0xFFFFu));
      atomicAdd(&start[4 * w + 2], (int)(lo >> 16));
      atomicAdd(&start[4 * w + 3], (int)(hi >> 16));
      atomicAdd(&before[4 * w], (int)(lo_before & 0xFFFFu));
      atomicAdd(&before[4 * w + 1], (int)(hi_before & 0xFFFFu));
      atomicAdd(&before[4 * w + 2], (int)(lo_before >> 16));
      atomicAdd(&before[4 * w + 3], (int)(hi_before >> 16));
    }
  }
  __syncthreads();
  scan_experts(start, E);
  if (b == 0)
    for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = start[e];
  for (int e = threadIdx.x; e < E; e += blockDim.x) before[e] += start[e];
  __syncthreads();
  place(id, t0, here, top_k, mask, before, positions, rows);
  // this block's share of the rows that no slot takes
  const int64_t lo = (int64_t)t0 * top_k, hi = lo + (int64_t)here * top_k;
  for (int64_t i = (lo > start[E] ? lo : start[E]) + threadIdx.x; i < hi; i += blockDim.x) rows[i] = -1;
}

template <int LG, int EPL>
void launch_choose(const void* logits, int ld, bool fp32, int T, int E, int top_k, bool renormalize, int* ids,
                   float* weights, int* offsets, int* rows, int* positions, uint8_t* counts, hipStream_t stream) {
  const dim3 grid((T + kTokens - 1) / kTokens);
  const int tokens = T < kTokens ? T : kTokens, threads = (tokens * LG + 63) / 64 * 64;
  const dim3 block(threads < 1024 ? threads : 1024);
  if (fp32)
    hipLaunchKernelGGL((route_kernel<LG, EPL, float>), grid, block, 0, stream, static_cast<const float*>(logits), ld, T,
                       E, top_k, (int)renormalize, ids, weights, offsets, rows, positions, counts);
  else
    hipLaunchKernelGGL((route_kernel<LG, EPL, _Float16>), grid, block, 0, stream, static_cast<const _Float16*>(logits),
                       ld, T, E, top_k, (int)renormalize, ids, weights, offsets, rows, positions, counts);
}

int blocks_of(int T) { return (T + kTokens - 1) / kTokens; }

size_t count_bytes(int T, int E) { return ((size_t)blocks_of(T) * ((E + 3) & ~3) + 15) & ~(size_t)15; }

}  // namespace

size_t route_workspace_bytes(int T, int E) {
  const int blocks = blocks_of(T);
  if (blocks <= 1) return 0;
  return count_bytes(T, E) + (blocks > kSumBlocks ? (size_t)(blocks + 1) * ((E + 3) & ~3) * 4 : 0);
}

hipError_t launch_route(const void* logits, int ld, bool fp32, int T, int E, int top_k, bool renormalize, int* ids,
                        float* weights, int* offsets, int* rows, int* positions, void* workspace, hipStream_t stream) {
  uint8_t* counts = static_cast<uint8_t*>(workspace);
#define AWQ_ROUTE(LG, EPL) \
  launch_choose<LG, EPL>(logits, ld, fp32, T, E, top_k, renormalize, ids, weights, offsets, rows, positions, counts, stream)
  if (E <= 8) AWQ_ROUTE(8, 1);
  else if (E <= 16) AWQ_ROUTE(8, 2);
  else if (E <= 32) AWQ_ROUTE(8, 4);
  else if (E <= 64) AWQ_ROUTE(8, 8);
  else if (E <= 128) AWQ_ROUTE(16, 8);
  else if (E <= 256) AWQ_ROUTE(16, 16);
  else if (E <= 512) AWQ_ROUTE(32, 16);
  else AWQ_ROUTE(64, 16);
#undef AWQ_ROUTE
  const int blocks = blocks_of(T);
  if (blocks > 1) {
    int* base = nullptr;
    const int words = (E + 3) / 4;
    const uint32_t* four = reinterpret_cast<const uint32_t*>(counts);
    if (blocks > kSumBlocks) {
      base = reinterpret_cast<int*>(counts + count_bytes(T, E));
      hipLaunchKernelGGL(route_sum_kernel, dim3(words), dim3(1024), 0, stream, four, blocks, words, base);
    }
    hipLaunchKernelGGL(route_place_kernel, dim3(blocks), dim3(words > 32 ? 1024 : 256), 0, stream, ids, T, E, top_k,
                       four, base, offsets, rows, positions);
  }
  return hipGetLastError();
}

}  // namespace awq
