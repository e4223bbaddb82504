// A few rows: the fused layer for 2-8 tokens, and expert rows in tiles of 4.
//
// Mathematics: awq_experts.hip's, with the exact integers q - z on the matrix
// cores and the group's scale on each 32-channel fp32 sum, so no weight is
// rounded.
//
// Bound: one memory round trip, then HBM.  v_mfma_f32_4x4x4_16b_f16 multiplies
// 16 independent 4 x 4 x 4 blocks: its blocks are 16 slices of 32 channels of
// the same rows, so lane (b, q) = (lane / 4, lane % 4) holds slice b of weight
// row q and of token q, and a wave's load reads 256 bytes of each of 4 rows.
// A workgroup owns two octets of weight rows (gated: an octet of gate rows and
// the octet of up rows they meet) and all of K; each of its waves takes S
// sub-chunks of 512 channels a round, with every load of a round in flight
// before any decoding.  The slices are summed across lanes in registers and the
// waves in LDS, in a fixed order; the last few threads apply the epilogue.
//
// Measured (us): 4 / 8 x 4096 -> 4096: 5.4 / 6.2; -> 11008: 9.6 / 12.2; -> 22016
// gated: 16.0 / 20.9 (2.9 / 2.3 TB/s); 4 tokens x 2 of 8 -> 22016 gated: 59 (4.3 TB/s).
#include "awq_epilogue.hpp"
#include "awq_launch_fused.hpp"

namespace awq {
namespace {

constexpr uint32_t kOutOfRange = 0x80000000u;  // a buffer offset past every resource: loads return 0
constexpr int kRows = 16;                      // weight rows per workgroup

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

// (What the loads need comes first, as plain arguments: the leading 16 words of
// the arguments are in registers when a wave starts.)
// TS: sets of 4 tokens; S: sub-chunks per wave and round; MULTI: K takes more
// than one round (a loop around the loads makes the compiler stage them less
// aggressively, so a single round is an instance of its own).
template <int TS, int S, int MAXW, bool ZP, bool MULTI, bool GROUPED>
__global__ __launch_bounds__(MAXW * 64) void few_kernel(const uint32_t* __restrict__ qweight,
                                                        const uint16_t* __restrict__ scales,
                                                        const uint32_t* __restrict__ qzeros,
                                                        const _Float16* __restrict__ xs, int N, int K, int ldx, int R,
                                                        int gshift, int gated, int groups, int rounds, int E,
                                                        ProductArgs p, float* __restrict__ part) {
  constexpr int RS = kRows / 4;
  __shared__ float red[MAXW][kRows][TS * 4];
  const int nw = blockDim.x >> 6;
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int b = lane >> 2, q = lane & 3;
  const int G = K >> gshift;
  const int width = gated ? N >> 1 : N;
  int grp = blockIdx.x;
  RowTile rt{0, 0, R};
  if constexpr (GROUPED) {
    // (the row tiles of an expert next to each other: its weights come from HBM once)
    const RowTiles tiles(p.offsets, E, R, TS * 4, 1);
    grp = blockIdx.x / max(tiles.total, 1);
    if (grp >= groups || tiles.total == 0) return;
    rt = tiles[blockIdx.x - grp * tiles.total];
  }
  const int n0 = grp * (gated ? 8 : kRows);  // first output column
  const size_t e = rt.expert;
  const DecodeConsts kc;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(qweight + e * N * (K >> 3), (uint32_t)N * (K >> 1));
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(scales + e * N * G, (uint32_t)N * G * 2);
  const __amdgpu_buffer_rsrc_t rz = make_rsrc(ZP ? qzeros + e * (N >> 3) * G : qweight,
                                              ZP ? (uint32_t)(N >> 3) * G * 4 : 0u);
  const __amdgpu_buffer_rsrc_t rx =
      GROUPED && p.rows ? make_rsrc(xs, (uint32_t)((p.x_rows - 1) * ldx + K) * 2)
                        : make_rsrc(xs + rt.row0 * (int64_t)ldx, (uint32_t)((rt.count - 1) * ldx + K) * 2);
  // the two octets; one past N lies past the resources and reads as 0
  uint32_t octet[2];
  octet[0] = n0 >> 3;
  octet[1] = gated ? (width + n0) >> 3 : octet[0] + 1;
  uint32_t xrow[TS];
#pragma unroll
  for (int ts = 0; ts < TS; ++ts) {
    const int m = 4 * ts + q;
    int r = min(m, rt.count - 1);
    if (GROUPED && p.rows) r = min(max(p.rows[rt.row0 + r] / p.slots_per_row, 0), p.x_rows - 1);
    xrow[ts] = m < rt.count ? (uint32_t)(r * ldx) * 2 : kOutOfRange;
  }

  float4_t acc[RS][TS];
#pragma unroll
  for (int r = 0; r < RS; ++r)
#pragma unroll
    for (int ts = 0; ts < TS; ++ts) acc[r][ts] = float4_t{0.f, 0.f, 0.f, 0.f};

  for (int round = 0; round < (MULTI ? rounds : 1); ++round) {
    u32x4 wv[S][RS], sv[S][2], xv[S][TS][4];
    uint32_t zv[S][2];
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int k0 = ((round * nw + wave) * S + s) * 512 + 32 * b;
      const bool kin = k0 < K;  // K is a multiple of 32: a slice is wholly in or out
      const int g = k0 >> gshift;
#pragma unroll
      for (int r = 0; r < RS; ++r) {
        const uint32_t row = octet[r >> 1] * 8 + 4 * (r & 1) + q;
        wv[s][r] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                       rw, kin && row < (uint32_t)N ? row * (K >> 1) + (k0 >> 1) : kOutOfRange, 0, 0));
      }
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const uint32_t at = octet[o] * G + g;
        sv[s][o] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, kin ? at * 16 : kOutOfRange, 0, 0));
        zv[s][o] = ZP ? __builtin_amdgcn_raw_buffer_load_b32(rz, kin ? at * 4 : kOutOfRange, 0, 0) : 0x88888888u;
      }
#pragma unroll
      for (int ts = 0; ts < TS; ++ts) {
        const uint32_t xo = kin ? xrow[ts] + 2 * k0 : kOutOfRange;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          xv[s][ts][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, xo, i * 16, 0));
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // every load of the round is in flight before any decoding
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int r = 0; r < RS; ++r) {
        const ZeroBias zb = zero_bias((zv[s][r >> 1] >> (4 * (4 * (r & 1) + q))) & 15u);
        float4_t tmp[TS];
#pragma unroll
        for (int ts = 0; ts < TS; ++ts) tmp[ts] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          half2_t d[4];
          decode_pairs(wv[s][r][i], zb, kc, d);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const half4_t a = {d[2 * h][0], d[2 * h][1], d[2 * h + 1][0], d[2 * h + 1][1]};
#pragma unroll
            for (int ts = 0; ts < TS; ++ts) {
              const half2_t x0 = as_half2(xv[s][ts][i][2 * h]), x1 = as_half2(xv[s][ts][i][2 * h + 1]);
              const half4_t x = {x0[0], x0[1], x1[0], x1[1]};
              tmp[ts] = __builtin_amdgcn_mfma_f32_4x4x4f16(a, x, tmp[ts], 0, 0, 0);
            }
          }
        }
        // register i of tmp is row 4 r + i: its scale for this slice's group
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int pos = 4 * (r & 1) + i;
          const uint32_t bits = (sv[s][r >> 1][pos >> 1] >> (16 * (pos & 1))) & 0xFFFFu;
          const float sc = (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
#pragma unroll
          for (int ts = 0; ts < TS; ++ts) acc[r][ts][i] += tmp[ts][i] * sc;
        }
      }
  }

  // Sum over the 16 slices (lane bits 2-5): the two lane-half swaps leave, in
  // 16-lane group g, register (0, 2, 1, 3)[g] summed over bits 4 and 5; two
  // DPP rotations within the 16 lanes add bits 3 and 2.
#pragma unroll
  for (int r = 0; r < RS; ++r)
#pragma unroll
    for (int ts = 0; ts < TS; ++ts) {
      const float a01 = swap_sum32(acc[r][ts][0], acc[r][ts][1]);
      const float a23 = swap_sum32(acc[r][ts][2], acc[r][ts][3]);
      float v = swap_sum16(a01, a23);
      v += row_rotate<0x128>(v);  // row_ror:8
      v += row_rotate<0x124>(v);  // row_ror:4
      const int g = lane >> 4;
      const int reg = g == 0 ? 0 : g == 1 ? 2 : g == 2 ? 1 : 3;
      if ((lane & 12) == 0) red[wave][4 * r + reg][4 * ts + q] = v;
    }
  __syncthreads();
  auto total = [&](int row, int m) __attribute__((always_inline)) {
    float sum = red[0][row][m];
    for (int i = 1; i < nw; ++i) sum += red[i][row][m];
    return sum;
  };
  const int outs = gated && !part ? 8 : kRows;
  for (int i = t; i < outs * TS * 4; i += nw * 64) {
    const int m = i / outs, row = i - m * outs;
    const int col = n0 + (gated ? row & 7 : row);
    if (m >= rt.count || col >= width) continue;
    const int64_t r = rt.row0 + m;
    const int n = gated && row >= 8 ? width + col : col;
    float v = total(row, m);
    if (p.bias) v += (float)p.bias[e * N + n];
    if (part) {  // raw sums, part[row][N]
      part[r * N + n] = v;
      continue;
    }
    v = activate(v, p.activation);
    if (gated) {
      float u = total(row + 8, m);
      if (p.bias) u += (float)p.bias[e * N + width + n];
      v *= u;
    }
    if (p.residual) v += (float)p.residual[r * p.ldr + col];
    p.y[r * p.ldy + col] = (_Float16)v;
  }
}

template <int TS, int S, int MAXW, bool ZP>
hipError_t launch_few_as(const PackedArgs& w, const ProductArgs& p, int gs, int nw, int rounds, float* part,
                         hipStream_t stream) {
  const int width = p.gated ? w.N / 2 : w.N, outs = p.gated ? 8 : kRows;
  const int groups = (width + outs - 1) / outs;
  const int slots = p.offsets ? row_tiles(p.R, w.E, TS * 4) : 1;
  auto kernel = rounds == 1 ? few_kernel<TS, S, MAXW, ZP, false, false> : few_kernel<TS, S, MAXW, ZP, true, false>;
  if constexpr (TS == 1) {
    if (p.offsets)
      kernel = rounds == 1 ? few_kernel<TS, S, MAXW, ZP, false, true> : few_kernel<TS, S, MAXW, ZP, true, true>;
  }
  hipLaunchKernelGGL(kernel, dim3((unsigned)(groups * slots)), dim3(nw * 64), 0, stream, w.qweight, w.scales, w.qzeros, p.x,
                     w.N, w.K, (int)p.ldx, p.R, gs, (int)p.gated, groups, rounds, w.E, p, part);
  return hipGetLastError();
}

// Sub-chunks per wave, waves and rounds: up to 4 rows two sub-chunks and up to
// 12 waves (124 registers), 5-8 rows at most 8 waves with two, or three once
// K needs more than 16 sub-chunks (one sub-chunk per wave, or more per wave on
// fewer waves, are 1-4% slower on the 7B shapes).
template <bool ZP>
hipError_t launch_few_zp(const PackedArgs& w, const ProductArgs& p, int gs, int rows, float* part, hipStream_t stream) {
  const int sub = (w.K + 511) / 512, maxw = rows <= 4 ? 12 : 8;
  const int s = rows <= 4 || sub <= 2 * maxw ? 2 : 3;
  int nw = (sub + s - 1) / s;
  if (nw > maxw) nw = maxw;
  const int rounds = (sub + nw * s - 1) / (nw * s);
  if (rows <= 4) return launch_few_as<1, 2, 12, ZP>(w, p, gs, nw, rounds, part, stream);
  return s == 2 ? launch_few_as<2, 2, 8, ZP>(w, p, gs, nw, rounds, part, stream)
                : launch_few_as<2, 3, 8, ZP>(w, p, gs, nw, rounds, part, stream);
}

}  // namespace

hipError_t launch_few(const PackedArgs& w, const ProductArgs& p, int gshift, int rows, float* part, hipStream_t stream) {
  // one tile holds all rows of a layer; experts' tiles have 4
  if (p.offsets ? rows != 4 : p.R > rows) return hipErrorInvalidValue;
  return w.qzeros ? launch_few_zp<true>(w, p, gshift, rows, part, stream)
                  : launch_few_zp<false>(w, p, gshift, rows, part, stream);
}

}  // namespace awq
