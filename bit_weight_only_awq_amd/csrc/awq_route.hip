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
// The sort is a counting sort without atomics on anything but bits: a token
// chooses an expert at most once, so the choices of 64 tokens for one expert
// are one 64-bit word with bit t set, and a slot's rank among its expert's
// slots is a population count.  Blocks of 256 tokens count their slots per
// expert; with more than one block a second launch adds the counts of the blocks before.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "awq_launch_fused.hpp"

namespace awq {
namespace {

constexpr int kTokens = 256;     // tokens per block
constexpr int kMaxExperts = 1024;

// Largest of v over groups of LG consecutive lanes.
template <int LG>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int d = 1; d < LG; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
template <int LG>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = 1; d < LG; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ float exp_below(float l, float m) { return l == m ? 1.0f : expf(l - m); }

// LG lanes per token, EPL consecutive logits per lane.
template <int LG, int EPL, typename T>
__device__ void choose(const T* __restrict__ logits, int64_t ld, int tokens, int E, int top_k, bool renormalize,
                       int* __restrict__ ids, float* __restrict__ weights) {
  const int lane = threadIdx.x & 63, l = lane & (LG - 1), base = lane & ~(LG - 1);
  const int per_pass = blockDim.x / LG;
  for (int t0 = 0; t0 < tokens; t0 += per_pass) {
    const int t = t0 + threadIdx.x / LG;
    const bool live = t < tokens;
    float v[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = l * EPL + i;
      v[i] = live && e < E ? (float)logits[t * ld + e] : -INFINITY;
      if (v[i] != v[i]) v[i] = -INFINITY;
    }
    float all = 0.0f, m = 0.0f, sum = 0.0f;
    for (int j = 0; j < top_k; ++j) {
      float mine = v[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) mine = fmaxf(mine, v[i]);
      const float best = group_max<LG>(mine);
      if (j == 0) {
        m = best;
#pragma unroll
        for (int i = 0; i < EPL; ++i) all += v[i] == -INFINITY ? 0.0f : exp_below(v[i], m);
        all = group_sum<LG>(all);
      }
      const bool any = best != -INFINITY;
      const unsigned long long has = __ballot(mine == best) >> base;
      const int owner = __builtin_ctzll(has | (1ull << 63));
      if (any) sum += exp_below(best, m);
      if (live && (any ? l == owner : l == 0)) {
        int at = -1;
        if (any) {
#pragma unroll
          for (int i = EPL - 1; i >= 0; --i)
            if (v[i] == best) at = i;
#pragma unroll
          for (int i = 0; i < EPL; ++i)
            if (i == at) v[i] = -INFINITY;
          at += l * EPL;
        }
        ids[(int64_t)t * top_k + j] = at;
        weights[(int64_t)t * top_k + j] = any ? exp_below(best, m) : 0.0f;
      }
    }
    if (live) {
      const float total = renormalize ? sum : all;
      __threadfence_block();
      for (int j = l; j < top_k; j += LG) {
        const int64_t s = (int64_t)t * top_k + j;
        weights[s] = total > 0.0f ? weights[s] / total : 0.0f;
      }
    }
  }
}

// The block's choices as bits: mask[e][w] bit b = token 64 w + b chose expert e.
__device__ void mark(const int* ids, int tokens, int E, int top_k, unsigned long long (*mask)[kTokens / 64]) {
  for (int i = threadIdx.x; i < E * (kTokens / 64); i += blockDim.x) (&mask[0][0])[i] = 0;
  __syncthreads();
  for (int s = threadIdx.x; s < tokens * top_k; s += blockDim.x) {
    const int e = ids[s], t = s / top_k;
    if (e >= 0) atomicOr(&mask[e][t >> 6], 1ull << (t & 63));
  }
  __syncthreads();
}

__device__ int count_of(const unsigned long long* m) {
  int n = 0;
#pragma unroll
  for (int w = 0; w < kTokens / 64; ++w) n += __popcll(m[w]);
  return n;
}

// start[e] (LDS) holds expert e's slots in all blocks: replaced by the sum over
// the experts below; start[E] the total.  One wave.
__device__ void scan_experts(int* start, int E) {
  if (threadIdx.x < 64) {
    int seen = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + threadIdx.x;
      const int n = e < E ? start[e] : 0;
      int sum = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(sum, d);
        if ((int)threadIdx.x >= d) sum += up;
      }
      if (e < E) start[e] = seen + sum - n;
      seen += __shfl(sum, 63);
    }
    if (threadIdx.x == 0) start[E] = seen;
  }
  __syncthreads();
}

// Positions and rows of the block's slots, from the masks and the place of
// the block's first slot of each expert.
__device__ void place(const int* ids, int t0, int tokens, int top_k, const unsigned long long (*mask)[kTokens / 64],
                      const int* first, int* __restrict__ positions, int* __restrict__ rows) {
  for (int s = threadIdx.x; s < tokens * top_k; s += blockDim.x) {
    const int e = ids[s], t = s / top_k;
    int at = -1;
    if (e >= 0) {
      at = first[e];
      for (int w = 0; w < (t >> 6); ++w) at += __popcll(mask[e][w]);
      at += __popcll(mask[e][t >> 6] & ((1ull << (t & 63)) - 1));
      rows[at] = t0 * top_k + s;
    }
    positions[(int64_t)t0 * top_k + s] = at;
  }
}

// One block: choices of kTokens tokens, and either the whole sort (one block
// in the grid) or the block's counts per expert.
template <int LG, int EPL, typename T>
__global__ __launch_bounds__(1024) void route_kernel(const T* __restrict__ logits, int ld, int tokens, int E, int top_k,
                                                     int renormalize, int* __restrict__ ids,
                                                     float* __restrict__ weights, int* __restrict__ offsets,
                                                     int* __restrict__ rows, int* __restrict__ positions,
                                                     int* __restrict__ counts) {
  __shared__ unsigned long long mask[kMaxExperts][kTokens / 64];
  __shared__ int start[kMaxExperts + 1];
  const int t0 = blockIdx.x * kTokens, here = min(kTokens, tokens - t0);
  int* my_ids = ids + (int64_t)t0 * top_k;
  choose<LG, EPL, T>(logits + (int64_t)t0 * ld, ld, here, E, top_k, renormalize != 0, my_ids,
                     weights + (int64_t)t0 * top_k);
  __syncthreads();
  mark(my_ids, here, E, top_k, mask);
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) counts[blockIdx.x * E + e] = count_of(mask[e]);
    return;
  }
  for (int e = threadIdx.x; e < E; e += blockDim.x) start[e] = count_of(mask[e]);
  __syncthreads();
  scan_experts(start, E);
  for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = start[e];
  place(my_ids, 0, here, top_k, mask, start, positions, rows);
  for (int i = start[E] + threadIdx.x; i < tokens * top_k; i += blockDim.x) rows[i] = -1;
}

__global__ __launch_bounds__(1024) void route_place_kernel(const int* __restrict__ ids, int tokens, int E, int top_k,
                                                           const int* __restrict__ counts, int* __restrict__ offsets,
                                                           int* __restrict__ rows, int* __restrict__ positions) {
  __shared__ unsigned long long mask[kMaxExperts][kTokens / 64];
  __shared__ int start[kMaxExperts + 1], before[kMaxExperts];
  const int t0 = blockIdx.x * kTokens, here = min(kTokens, tokens - t0);
  const int* my_ids = ids + (int64_t)t0 * top_k;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int sum = 0, mine = 0;
    for (int b = 0; b < (int)gridDim.x; ++b) {
      if (b == (int)blockIdx.x) mine = sum;
      sum += counts[b * E + e];
    }
    start[e] = sum;
    before[e] = mine;
  }
  mark(my_ids, here, E, top_k, mask);
  scan_experts(start, E);
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = start[e];
  for (int e = threadIdx.x; e < E; e += blockDim.x) before[e] += start[e];
  __syncthreads();
  place(my_ids, t0, here, top_k, mask, before, positions, rows);
  // this block's share of the rows that no slot takes
  const int64_t lo = (int64_t)t0 * top_k, hi = lo + (int64_t)here * top_k;
  for (int64_t i = (lo > start[E] ? lo : start[E]) + threadIdx.x; i < hi; i += blockDim.x) rows[i] = -1;
}

template <int LG, int EPL>
void launch_choose(const void* logits, int ld, bool fp32, int T, int E, int top_k, bool renormalize, int* ids,
                   float* weights, int* offsets, int* rows, int* positions, int* counts, hipStream_t stream) {
  const dim3 grid((T + kTokens - 1) / kTokens);
  if (fp32)
    hipLaunchKernelGGL((route_kernel<LG, EPL, float>), grid, dim3(1024), 0, stream, static_cast<const float*>(logits),
                       ld, T, E, top_k, (int)renormalize, ids, weights, offsets, rows, positions, counts);
  else
    hipLaunchKernelGGL((route_kernel<LG, EPL, _Float16>), grid, dim3(1024), 0, stream,
                       static_cast<const _Float16*>(logits), ld, T, E, top_k, (int)renormalize, ids, weights, offsets,
                       rows, positions, counts);
}

}  // namespace

size_t route_workspace_bytes(int T, int E) {
  const size_t blocks = ((size_t)T + kTokens - 1) / kTokens;
  return blocks > 1 ? blocks * E * 4 : 0;
}

hipError_t launch_route(const void* logits, int ld, bool fp32, int T, int E, int top_k, bool renormalize, int* ids,
                        float* weights, int* offsets, int* rows, int* positions, void* workspace, hipStream_t stream) {
  int* counts = static_cast<int*>(workspace);
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
  if (T > kTokens)
    hipLaunchKernelGGL(route_place_kernel, dim3((T + kTokens - 1) / kTokens), dim3(1024), 0, stream, ids, T, E, top_k,
                       counts, offsets, rows, positions);
  return hipGetLastError();
}

}  // namespace awq
