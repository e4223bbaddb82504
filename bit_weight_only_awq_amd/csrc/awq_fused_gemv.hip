// One row at a time: the fused layer for a single token, expert rows that (nearly)
// all have an expert of their own, and the weighted sum of a token's few slots.
//
// Mathematics: awq_experts.hip's, with the exact integers q - z in fp16 dot
// products (v_dot2_f32_f16, fp32 sums) and the group's scale on each
// 32-channel sum, so no weight is rounded.
//
// Bound: HBM, each packed byte used once, and at these sizes the launch and one
// memory round trip.  A group of ROWS weight rows (gated: half of them gate
// rows and half the up rows they meet, so one workgroup holds both factors of
// its outputs) is read by NW waves, each lane one 32-channel chunk of every row
// per pass, every load of a pass in flight before any decoding; the row sums
// meet in registers across the wave and in LDS across the waves, in a fixed
// order, and the last few threads apply the epilogue.  The combining kernel
// lays the token's slots end to end: a chunk belongs to one slot, whose
// expert's rows it reads and whose weight multiplies its sum, so the weighted
// sum over experts is the same reduction and needs no second launch.
//
// Measured: 4096 -> 4096: 3.7 us, with residual 3.8; 4096 -> 22016 gated: 10.1-10.5
// us, 4.5-4.6 TB/s; one token x 2 of 8, the same layer: 20.2-20.9 us, 4.5-4.6 TB/s;
// combined 11008 -> 4096: 14.1 us, 3.3 TB/s.  Bytes read: 1.00-1.01 of the packed weights.
#include "awq_epilogue.hpp"
#include "awq_launch_fused.hpp"

namespace awq {
namespace {

// Row `r` of the sorted order: the expert whose range holds it, or -1.  `ends`:
// the ends of the first 64 experts' ranges, one per lane, and `first`, where the
// first of them begins (loaded early).
__device__ __forceinline__ int range_ends(const int* __restrict__ offsets, int E, int e0) {
  const int e = e0 + __lane_id();
  return e < E ? offsets[e + 1] : 0;
}
__device__ __forceinline__ int expert_of_row(const int* __restrict__ offsets, int E, int first, int ends, int r) {
  if (r < first) return -1;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const unsigned long long past = __ballot((e0 == 0 ? ends : range_ends(offsets, E, e0)) > r);
    if (past != 0) return e0 + __builtin_ctzll(past);
  }
  return -1;
}

// One chunk (32 channels) of ROWS weight rows: the loads of a lane.
template <int ROWS>
struct Chunk {
  u32x4 w[ROWS], x[4];
  uint32_t s[ROWS / 2], z[2];
};

// Sums of the chunk: q - z against x in two partial dot products, times the scale.
template <int ROWS, bool ZP>
__device__ __forceinline__ void add_chunk(float (&acc)[ROWS], const Chunk<ROWS>& c, const int (&zshift)[2], float weight,
                                          const DecodeConsts& kc) {
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int part = r / (ROWS / 2), i = r % (ROWS / 2);
    const ZeroBias b = zero_bias(ZP ? (c.z[part] >> (zshift[part] + 4 * i)) & 15u : 8u);
    float p0 = 0.0f, p1 = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      half2_t d[4];
      decode_pairs(c.w[r][k], b, kc, d);
      p0 = __builtin_amdgcn_fdot2(d[0], as_half2(c.x[k][0]), p0, false);
      p1 = __builtin_amdgcn_fdot2(d[1], as_half2(c.x[k][1]), p1, false);
      p0 = __builtin_amdgcn_fdot2(d[2], as_half2(c.x[k][2]), p0, false);
      p1 = __builtin_amdgcn_fdot2(d[3], as_half2(c.x[k][3]), p1, false);
    }
    const uint32_t bits = (c.s[r >> 1] >> (16 * (r & 1))) & 0xFFFFu;
    acc[r] += (p0 + p1) * ((float)__builtin_bit_cast(_Float16, (uint16_t)bits) * weight);
  }
}

// The wave's sum of row `row` (below) over its lanes.
template <int ROWS>
__device__ __forceinline__ float wave_sum(const float (&acc)[ROWS]) {
  if constexpr (ROWS == 8)
    return wave_reduce_oct_rows(acc);
  else
    return wave_reduce_quad_rows(acc);
}
template <int ROWS>
__device__ __forceinline__ int wave_sum_row(int lane) {
  return ROWS == 8 ? (lane >> 4) + 4 * ((lane >> 3) & 1) : lane >> 4;
}

// The ROWS weight rows of a group are two runs of ROWS / 2: n0 .. and n1 ..
// (plain: the next ROWS / 2; gated: the same outputs' up rows).  A run lies
// within one octet of rows, so its scales are one load and its zero points one word.
template <int ROWS>
struct Runs {
  const u32x4* w[2];
  const uint16_t* s[2];
  const uint32_t* z[2];
  int zshift[2];
};
template <int ROWS, bool ZP>
__device__ __forceinline__ Runs<ROWS> runs_of(const uint32_t* qweight, const uint16_t* scales, const uint32_t* qzeros,
                                              size_t expert, int N, int K, int G, int n0, int n1) {
  Runs<ROWS> r;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int n = p ? n1 : n0;
    r.w[p] = reinterpret_cast<const u32x4*>(qweight + (expert * N + n) * (size_t)(K >> 3));
    r.s[p] = scales + expert * N * G + scale_index(n, 0, G);
    r.z[p] = ZP ? qzeros + expert * (N >> 3) * G + zero_word_index(n, 0, G) : nullptr;
    r.zshift[p] = 4 * (n & 7);
  }
  return r;
}

// The loads of chunk c (32 channels from 32 c) of one slot.
template <int ROWS, bool ZP>
__device__ __forceinline__ void load_chunk(Chunk<ROWS>& ck, const Runs<ROWS>& r, const u32x4* __restrict__ x, int c,
                                           int K, int gshift) {
  const int grp = (c << 5) >> gshift;
  const size_t row_u4 = (size_t)(K >> 5);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    if constexpr (ROWS == 8) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(r.s[p] + (size_t)grp * 8);
      ck.s[2 * p] = v[0];
      ck.s[2 * p + 1] = v[1];
    } else {
      ck.s[p] = *reinterpret_cast<const uint32_t*>(r.s[p] + (size_t)grp * 8);
    }
    ck.z[p] = ZP ? r.z[p][grp] : 0u;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) ck.x[i] = x[(size_t)c * 4 + i];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) ck.w[i] = r.w[i / (ROWS / 2)][(size_t)(i % (ROWS / 2)) * row_u4 + c];
}

// Within each group of 64 workgroups the row groups are transposed, so that the
// outputs of a 128-byte line come from one XCD (workgroups are dealt to the 8
// XCDs in turn); a ragged last group keeps the dealt order.
__device__ __forceinline__ int placed(int b, int n) {
  return b < (n & ~63) ? (b & ~63) | ((b & 7) << 3) | ((b >> 3) & 7) : b;
}

// (The arguments that the first addresses need come first: the leading 16
// words of the arguments are in registers when a wave starts.)
template <int NW, bool ZP, int ROWS, int QPW, bool GROUPED>
__global__ __launch_bounds__(NW * QPW * 64) void fused_gemv_kernel(
    const _Float16* __restrict__ x, const uint32_t* __restrict__ qweight, const uint16_t* __restrict__ scales,
    const uint32_t* __restrict__ qzeros, int N, int K, int gshift, int width, int groups, const ProductArgs p, int E) {
  __shared__ float red[QPW][NW][ROWS];
  const int lane = threadIdx.x & 63, wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = QPW == 1 ? 0 : wave_all / NW, wave = wave_all - part * NW;
  const bool gated = width < N;
  const int outs = gated ? ROWS / 2 : ROWS;  // outputs per group
  const int slot = GROUPED ? blockIdx.x / groups : 0, b = GROUPED ? blockIdx.x - slot * groups : blockIdx.x;
  const int g0 = (placed(b, groups) * QPW + part) * outs;  // first output of the group
  const int n0 = min(g0, width - outs), n1 = gated ? width + n0 : n0 + ROWS / 2;
  size_t expert = 0;
  const _Float16* xr = x;
  if constexpr (GROUPED) {
    // (the source row is looked up beside the expert)
    const int ends = range_ends(p.offsets, E, 0), first = p.offsets[0];
    int r = slot;
    if (p.rows) r = min(max(p.rows[slot] / p.slots_per_row, 0), p.x_rows - 1);
    const int e = expert_of_row(p.offsets, E, first, ends, slot);
    if (e < 0) return;
    expert = e;
    xr = x + r * p.ldx;
  }
  const DecodeConsts kc;
  const Runs<ROWS> runs = runs_of<ROWS, ZP>(qweight, scales, qzeros, expert, N, K, K >> gshift, n0, n1);
  float acc[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) acc[r] = 0.0f;
  for (int c = wave * 64 + lane; c < K >> 5; c += NW * 64) {
    Chunk<ROWS> ck;
    load_chunk<ROWS, ZP>(ck, runs, reinterpret_cast<const u32x4*>(xr), c, K, gshift);
    __builtin_amdgcn_sched_barrier(0);  // every load before any decoding
    add_chunk<ROWS, ZP>(acc, ck, runs.zshift, 1.0f, kc);
  }
  const float total = wave_sum<ROWS>(acc);
  if (lane % (64 / ROWS) == 0) red[part][wave][wave_sum_row<ROWS>(lane)] = total;
  __syncthreads();
  const int q = threadIdx.x / outs, i = threadIdx.x - q * outs;
  const int n = (placed(b, groups) * QPW + q) * outs + i;
  if (q >= QPW || n >= width) return;
  float v = red[q][0][i], u = gated ? red[q][0][ROWS / 2 + i] : 0.0f;
#pragma unroll
  for (int w = 1; w < NW; ++w) {
    v += red[q][w][i];
    if (gated) u += red[q][w][ROWS / 2 + i];
  }
  if (p.bias) {
    v += (float)p.bias[expert * N + n];
    if (gated) u += (float)p.bias[expert * N + width + n];
  }
  v = activate(v, p.activation);
  if (gated) v *= u;
  if (p.residual) v += (float)p.residual[slot * p.ldr + n];
  p.y[slot * p.ldy + n] = (_Float16)v;
}

constexpr int kMaxSlots = 64;

template <int NW, bool ZP, int ROWS>
__global__ __launch_bounds__(NW * 64) void combine_gemv_kernel(
    const _Float16* __restrict__ x, const uint32_t* __restrict__ qweight, const uint16_t* __restrict__ scales,
    const uint32_t* __restrict__ qzeros, int N, int K, int gshift, int groups, const CombineArgs c, const ProductArgs p,
    int E) {
  __shared__ float red[NW][ROWS];
  __shared__ int slot_expert[kMaxSlots];
  __shared__ float slot_weight[kMaxSlots];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x / groups, b = blockIdx.x - t * groups;
  const int n0 = placed(b, groups) * ROWS;
  const int chunks = K >> 5, G = K >> gshift;
  // waves to slots: `side` of them share a slot's chunks, `sets` slots at a time
  const int side = c.top_k >= NW ? 1 : NW / c.top_k, sets = NW / side;
  const int ends = range_ends(p.offsets, E, 0), first = p.offsets[0];
  const int rows = lane < c.top_k ? c.positions[(int64_t)t * c.top_k + lane] : -1;
  const float weights = lane < c.top_k ? c.weights[(int64_t)t * c.top_k + lane] : 0.0f;
  const DecodeConsts kc;
  float acc[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) acc[r] = 0.0f;
  for (int j = wave / side; j < c.top_k && wave < side * sets; j += sets) {
    const int row = __builtin_amdgcn_readlane(rows, j);
    const float weight = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weights), j));
    const int e = row < 0 || row >= p.R ? -1 : expert_of_row(p.offsets, E, first, ends, row);
    if (wave % side == 0 && lane == 0) {
      slot_expert[j] = e;
      slot_weight[j] = weight;
    }
    if (e < 0) continue;
    const Runs<ROWS> runs = runs_of<ROWS, ZP>(qweight, scales, qzeros, e, N, K, G, n0, n0 + ROWS / 2);
    const u32x4* xr = reinterpret_cast<const u32x4*>(x + (int64_t)row * p.ldx);
    for (int ch = wave % side * 64 + lane; ch < chunks; ch += side * 64) {
      Chunk<ROWS> ck;
      load_chunk<ROWS, ZP>(ck, runs, xr, ch, K, gshift);
      __builtin_amdgcn_sched_barrier(0);
      add_chunk<ROWS, ZP>(acc, ck, runs.zshift, weight, kc);
    }
  }
  const float total = wave_sum<ROWS>(acc);
  if (lane % (64 / ROWS) == 0) red[wave][wave_sum_row<ROWS>(lane)] = total;
  __syncthreads();
  if (threadIdx.x >= ROWS) return;
  const int n = n0 + threadIdx.x;
  float v = red[0][threadIdx.x];
#pragma unroll
  for (int w = 1; w < NW; ++w) v += red[w][threadIdx.x];
  if (p.bias)
    for (int j = 0; j < c.top_k; ++j)
      if (slot_expert[j] >= 0) v += slot_weight[j] * (float)p.bias[(size_t)slot_expert[j] * N + n];
  if (c.residual) v += (float)c.residual[t * c.ldr + n];
  c.y[t * c.ldy + n] = (_Float16)v;
}

// Waves per row group: one 32-channel chunk per lane up to 8 waves, 12 past
// 512 chunks.
int gemv_waves(int chunks) { return chunks > 8 * 64 ? 12 : (chunks + 63) / 64; }

template <bool ZP, int ROWS>
hipError_t launch_gemv_rows(const PackedArgs& w, const ProductArgs& p, int gs, hipStream_t stream) {
  const int nw = gemv_waves(w.K >> 5), width = p.gated ? w.N / 2 : w.N, outs = p.gated ? ROWS / 2 : ROWS;
#define AWQ_FUSED_GEMV(W)                                                                                              \
  case W: {                                                                                                            \
    constexpr int QPW = ROWS == 4 && W <= 8 ? 2 : 1;                                                                   \
    const int groups = (width / outs + QPW - 1) / QPW;                                                                 \
    const auto kernel =                                                                                                \
        p.offsets ? fused_gemv_kernel<W, ZP, ROWS, QPW, true> : fused_gemv_kernel<W, ZP, ROWS, QPW, false>;            \
    hipLaunchKernelGGL(kernel, dim3((unsigned)(groups * p.R)), dim3(W * QPW * 64), 0, stream, p.x, w.qweight,          \
                       w.scales, w.qzeros, w.N, w.K, gs, width, groups, p, w.E);                                       \
    break;                                                                                                             \
  }
  switch (nw) {
    AWQ_FUSED_GEMV(1)
    AWQ_FUSED_GEMV(2)
    AWQ_FUSED_GEMV(3)
    AWQ_FUSED_GEMV(4)
    AWQ_FUSED_GEMV(5)
    AWQ_FUSED_GEMV(6)
    AWQ_FUSED_GEMV(7)
    AWQ_FUSED_GEMV(8)
    AWQ_FUSED_GEMV(12)
    default: return hipErrorInvalidValue;
  }
#undef AWQ_FUSED_GEMV
  return hipGetLastError();
}

template <bool ZP, int ROWS>
hipError_t launch_combine_rows(const PackedArgs& w, const ProductArgs& p, const CombineArgs& c, int gs, int nw,
                               hipStream_t stream) {
  const int groups = w.N / ROWS;
#define AWQ_COMBINE_GEMV(W)                                                                                       \
  case W:                                                                                                         \
    hipLaunchKernelGGL((combine_gemv_kernel<W, ZP, ROWS>), dim3((unsigned)(groups * c.T)), dim3(W * 64), 0, stream, \
                       p.x, w.qweight, w.scales, w.qzeros, w.N, w.K, gs, groups, c, p, w.E);                      \
    break;
  switch (nw) {
    AWQ_COMBINE_GEMV(1)
    AWQ_COMBINE_GEMV(2)
    AWQ_COMBINE_GEMV(3)
    AWQ_COMBINE_GEMV(4)
    AWQ_COMBINE_GEMV(6)
    AWQ_COMBINE_GEMV(8)
    AWQ_COMBINE_GEMV(12)
    AWQ_COMBINE_GEMV(16)
    default: return hipErrorInvalidValue;
  }
#undef AWQ_COMBINE_GEMV
  return hipGetLastError();
}

// Waves of a combining workgroup: one 32-channel chunk per lane for every slot,
// up to 16.
int combine_waves(int chunks, int top_k) {
  const int want = (chunks + 63) / 64 * top_k;
  for (int w : {1, 2, 3, 4, 6, 8, 12})
    if (want <= w) return w;
  return 16;
}

}  // namespace

// Groups of 8 weight rows halve the loads of x per packed byte, but make half
// as many workgroups.  For rows out they pay from ~32 waves per compute unit
// (two 4096 -> 22016 experts, 43: 21.1 us against 23.1; one 4096 -> 22016 layer,
// 21: 11.4 against 11.6; 4096 x 4096: 4.9 against 4.2); combining, whose
// workgroups are larger, from ~16 (two 11008 -> 4096 experts, 24: 15.6 us
// against 17.1; six 1408 -> 2048 experts, 5: 7.7 against 7.2).
hipError_t launch_fused_gemv(const PackedArgs& w, const ProductArgs& p, int gshift, hipStream_t stream) {
  const bool o = (int64_t)w.N / 8 * p.R * gemv_waves(w.K >> 5) >= 32 * 256;
  if (w.qzeros)
    return o ? launch_gemv_rows<true, 8>(w, p, gshift, stream) : launch_gemv_rows<true, 4>(w, p, gshift, stream);
  return o ? launch_gemv_rows<false, 8>(w, p, gshift, stream) : launch_gemv_rows<false, 4>(w, p, gshift, stream);
}

hipError_t launch_combine_gemv(const PackedArgs& w, const ProductArgs& p, const CombineArgs& c, int gshift,
                               hipStream_t stream) {
  const int nw = combine_waves(w.K >> 5, c.top_k);
  const bool o = (int64_t)w.N / 8 * c.T * nw >= 16 * 256;
  if (w.qzeros)
    return o ? launch_combine_rows<true, 8>(w, p, c, gshift, nw, stream)
             : launch_combine_rows<true, 4>(w, p, c, gshift, nw, stream);
  return o ? launch_combine_rows<false, 8>(w, p, c, gshift, nw, stream)
           : launch_combine_rows<false, 4>(w, p, c, gshift, nw, stream);
}

}  // namespace awq
