// Weight-stream bound products (from a few rows, or two per expert, to where the
// matrix-core tiles take less time): tiles of up to XR rows x 32 CW weight rows,
// with every operand flowing through a ring of LDS stages.
//
// Mathematics: awq_experts.hip's.  The matrix cores multiply the exact integers
// q - z, and the group's scale multiplies the fp32 sum once per group and output
// (16 multiply-adds per 32 x 32 tile in place of four packed multiplies per
// packed word): no weight is rounded.  A lane holds 32 channels of a 64-channel
// block; with groups of 32 the lane halves, whose channels then lie in different
// groups, exchange every other word first.
//
// Bound: HBM, the packed weights once, and what a compute unit takes in: a load
// whose 64 lanes touch 32 rows of 32 bytes runs at 37 bytes/ns per compute
// unit, one that reads 128 or 256 bytes of each row at 120.  So both
// operands go straight into a ring of LDS stages (buffer-to-LDS loads, whole
// 128-byte lines of packed words, 512 bytes of each row of X), D - 1 stages
// ahead, with one counted wait and one barrier per stage; each wave multiplies
// the 32 weight rows it loaded with rows of X shared by the CW waves of a
// stage.  KW waves split a stage's channels and their sums meet in LDS at the
// end; where the tiles are too few for the chip, K is split across workgroups
// as well, into fp32 partial sums that a second kernel adds in order.  Deeper
// rings (3 and 4 stages of 256 channels, or of 128) measure the same: with one
// workgroup per compute unit a stage's decoding and products take about as long
// as its loads.
//
// Measured: 48 tokens x 6 of 64, 2048 -> 2816 gated: 46.6 us, 4.1 TB/s of the
// packed weights (floor 37.0), in groups of 64: 51.5; 64 x 4096 -> 4096: 9.8 us; 13
// x 11008 -> 4096 with its second launch: 16.2; 61 x 4096 -> 11008, groups of 64:
// 18.2 (5.0), of 32: 22.3.
#include "awq_epilogue.hpp"
#include "awq_launch_fused.hpp"

namespace awq {
namespace {

constexpr uint32_t kOutOfRange = 0x80000000u;  // a buffer offset past every resource: loads return 0

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

// 16 bytes per lane from `rsrc` at the lane's offset plus a common one to LDS, lane after lane.
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t rsrc, char* to, uint32_t off, uint32_t all) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)to, 16, off, all, 0, 0);
}

// Group sizes: 0: 32; 1: 64; 2: 128 and 256.  SC: channels of a wave's stage.
// TAIL: the last stage runs past K.
template <bool ZP, bool TAIL, int GROUP, int XR, int CW, int KW, int D, int SC>
__global__ __launch_bounds__(CW* KW * 64) void stream_kernel(PackedArgs w, ProductArgs p, int gshift, int tiles_n,
                                                             int stages_per_split, float* __restrict__ part) {
  constexpr int WAVES = CW * KW, COLS = 32 * CW, NBLK = SC / 64;
  constexpr int RT = (XR + 31) / 32, XT = XR < 32 ? XR : 32;  // 32-row tiles; rows a fragment read wraps at
  constexpr int XROW = SC * 2, WROW = SC / 2;                 // bytes of a row of X and of W in a stage
  constexpr int XL = 1024 / XROW, WL = 1024 / WROW;           // rows of one load
  constexpr int XU = XR / (XL * CW), WU = 32 / WL;            // loads per wave and stage
  constexpr int NS = GROUP == 2 ? SC / 128 : NBLK;            // groups of a lane's weights in a stage
  constexpr int LOADS = XU + WU + NS * (ZP ? 2 : 1);          // vector loads of a stage
  constexpr int IN_FLIGHT = (D - 2) * LOADS;                  // loads of the stages after the next
  constexpr int X_BYTES = KW * XR * XROW, SLOT = X_BYTES + WAVES * 32 * WROW;
  // the sums leave through the ring's first stage
  constexpr int PITCH = KW * 32 * (COLS + 8) * 4 <= SLOT ? COLS + 8 : COLS;
  static_assert(KW * 32 * PITCH * 4 <= SLOT, "the sums fit a stage");
  // one array per stage, so that the wait before an LDS read covers only the
  // loads into the stage being read
  __shared__ __attribute__((aligned(1024))) char r0[SLOT], r1[SLOT], r2[D > 2 ? SLOT : 16];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cw = wave % CW, kw = wave / CW;
  const int fi = lane & 31, fh = lane >> 5;
  const int K = w.K, G = K >> gshift;
  const bool gated = p.gated;
  const int width = gated ? w.N >> 1 : w.N;
  const DecodeConsts kc;

  const RowTiles row_tiles(p.offsets, w.E, p.R, XR, 1);
  const int tiles = row_tiles.total * tiles_n, split = blockIdx.y;
  if ((int)blockIdx.x >= tiles) return;
  // consecutive tiles on one XCD: row tiles of an expert next to each other, so
  // that its weights are read from HBM once
  const int tile = xcd_contiguous_tile(blockIdx.x, tiles);
  const int tn = row_tiles.total == 1 ? tile : tile / row_tiles.total;  // (some tile: total > 0)
  const RowTile t = row_tiles[tile - tn * row_tiles.total];
  const int n0 = tn * (gated ? COLS / 2 : COLS);  // first output column
  const int nstages = (K + SC * KW - 1) / (SC * KW);
  const int s0 = split * stages_per_split, s1 = min(nstages, s0 + stages_per_split);

  // X: load i of this wave brings XL rows, SC channels of wave group kb; chunk
  // c of row r goes to slot c ^ (r % 16), so that fragment reads touch every bank once
  const void* xbase = p.rows ? p.x : p.x + t.row0 * p.ldx;
  const uint32_t xbytes = (uint32_t)((p.rows ? p.x_rows : t.count) * (int)p.ldx) * 2;
  uint32_t xoff[XU];
  int xch[XU];  // the load's first channel within the stage
#pragma unroll
  for (int i = 0; i < XU; ++i) {
    const int q = wave * XU + i, kb = q / (XR / XL), row = XL * (q % (XR / XL)) + lane / (64 / XL);
    int r = row;
    if (p.rows) r = min(max(p.rows[t.row0 + min(row, t.count - 1)] / p.slots_per_row, 0), p.x_rows - 1);
    xch[i] = kb * SC + 8 * ((lane & (64 / XL - 1)) ^ (row & 15));
    xoff[i] = row < t.count ? (uint32_t)(r * (int)p.ldx + xch[i]) * 2 : kOutOfRange;
  }
  // W: load i of this wave brings WL of its 32 weight rows (gated: 16 gate rows,
  // then the 16 up rows they meet), SC channels; chunk c (32 channels) of row r
  // goes to slot c ^ (r's place among the rows that share its banks)
  auto weight_row = [&](int i) __attribute__((always_inline)) {  // (rows past N: the last one again, never stored)
    return min(gated ? (i < 16 ? 0 : width - 16) + n0 + 16 * cw + i : n0 + 32 * cw + i, w.N - 1);
  };
  auto wswz = [&](int row) __attribute__((always_inline)) { return SC == 256 ? (row >> 1) & 7 : (row >> 2) & 3; };
  const size_t e = t.expert;
  const void* wbase = w.qweight + e * w.N * (K >> 3);
  const void* sbase = w.scales + e * w.N * G;
  const void* zbase = ZP ? w.qzeros + e * (w.N >> 3) * G : w.qweight;
  const uint32_t wbytes = (uint32_t)w.N * (K >> 1), sbytes = (uint32_t)w.N * G * 2, zbytes = (uint32_t)(w.N >> 3) * G * 4;
  uint32_t woff[WU];
  int wch[WU];  // the load's first channel within the wave's SC
#pragma unroll
  for (int i = 0; i < WU; ++i) {
    const int row = WL * i + lane / (64 / WL);
    wch[i] = 32 * ((lane & (64 / WL - 1)) ^ wswz(row));
    woff[i] = (uint32_t)weight_row(row) * (K >> 1) + ((kw * SC + wch[i]) >> 1);
  }
  // scales and zero points: lane (i, h) = (lane % 32, lane / 32) holds row i's, in registers
  const int wr = weight_row(fi);
  const uint32_t srow = (uint32_t)((wr >> 3) * G), spart = (uint32_t)(wr & 7) * 2;
  const int zshift = 4 * (wr & 7);

  auto ring = [&](int c) __attribute__((always_inline)) { return c == 0 ? r0 : c == 1 ? r1 : r2; };
  struct Groups {
    uint32_t s[NS], z[NS];
  };
  // Stage s into slot c (a constant at every call site).  The stage goes into
  // the scalar offset, which the range check leaves out: channels past K are
  // sent out of range by their lane offset, and past the slice's last stage
  // the buffers are empty (their loads read 0 and cost no traffic).
  auto load = [&](int s, int c, Groups& x) __attribute__((always_inline)) {
    const bool live = s < s1;
    const int k = s * (SC * KW);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(xbase, live ? xbytes : 0u), rw = make_rsrc(wbase, live ? wbytes : 0u);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(sbase, live ? sbytes : 0u), rz = make_rsrc(zbase, live ? zbytes : 0u);
#pragma unroll
    for (int i = 0; i < WU; ++i)
      load_lds(rw, ring(c) + X_BYTES + (wave * WU + i) * 1024,
               TAIL && k + kw * SC + wch[i] >= K ? kOutOfRange : woff[i], k >> 1);
#pragma unroll
    for (int i = 0; i < XU; ++i)
      load_lds(rx, ring(c) + (wave * XU + i) * 1024, TAIL && k + xch[i] >= K ? kOutOfRange : xoff[i], 2 * k);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      if constexpr (GROUP == 0) {
        const uint32_t at = srow + (min(k + kw * SC + 64 * i + 32 * fh, K - 1) >> gshift);
        x.s[i] = __builtin_amdgcn_raw_buffer_load_b16(rs, at * 16 + spart, 0, 0);
        x.z[i] = ZP ? __builtin_amdgcn_raw_buffer_load_b32(rz, at * 4, 0, 0) : 0u;
      } else {
        const int g = min(k + kw * SC + (GROUP == 2 ? 128 : 64) * i, K - 1) >> gshift;
        x.s[i] = __builtin_amdgcn_raw_buffer_load_b16(rs, srow * 16 + spart, g * 16, 0);
        x.z[i] = ZP ? __builtin_amdgcn_raw_buffer_load_b32(rz, srow * 4, g * 4, 0) : 0u;
      }
    }
  };

  float16_t acc[RT];
#pragma unroll
  for (int a = 0; a < RT; ++a) acc[a] = float16_t(0.0f);

  // One stage, software-pipelined by hand (a SIMD has only a wave or two to
  // hide latency behind): the fragments of a 64-channel block are read from
  // LDS while the block before it is decoded and multiplied, and a group's
  // scale is applied while the next group multiplies.
  u32x4 wv[NBLK];
  half8_t af[2][4][RT];
  // slice j's chunk of 8 channels within the block, for X and W alike
  auto chunk_of = [&](int j) __attribute__((always_inline)) { return GROUP == 0 ? 2 * j + fh : 4 * fh + j; };
  auto read_block = [&](int c, int b) __attribute__((always_inline)) {
    const char* xs = ring(c) + kw * XR * XROW;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int a = 0; a < RT; ++a)
        af[b & 1][j][a] = *reinterpret_cast<const half8_t*>(xs + (32 * a + (fi & (XT - 1))) * XROW +
                                                            16 * ((8 * b + chunk_of(j)) ^ (fi & 15)));
  };
  auto begin = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < NBLK; ++b)
      wv[b] = *reinterpret_cast<const u32x4*>(ring(c) + X_BYTES + wave * 32 * WROW + fi * WROW +
                                              16 * ((2 * b + fh) ^ wswz(fi)));
    read_block(c, 0);
  };
  // (All 16 sums of a tile are added up, also where it has 16 rows only: with
  // half of a matrix instruction's result unused, the compiler let another's
  // overlap that half, and sums came out wrong.)
  float16_t tmp[2][RT];
  auto apply = [&](int g, float s) __attribute__((always_inline)) {
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][r] = __builtin_fmaf(tmp[g & 1][a][r], s, acc[a][r]);
  };
  auto scale_of = [&](uint32_t bits) __attribute__((always_inline)) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  };
  auto compute = [&](int c, const Groups& x) __attribute__((always_inline)) {
    ZeroBias zb;
    float scale[2];  // of the last two groups
#pragma unroll
    for (int b = 0; b < NBLK; ++b) {
      if (b + 1 < NBLK) read_block(c, b + 1);
      __builtin_amdgcn_sched_barrier(0);
      uint32_t z[2], sb[2], w[4];  // the block's two groups (groups of 32), or its one in [0]
      {
        const int g = GROUP == 2 ? b / 2 : b;
        z[0] = ZP ? (x.z[g] >> zshift) & 15u : 8u;
        sb[0] = x.s[g];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = wv[b][j];
      }
      if constexpr (GROUP == 0) {
        // (words 4 h .. 4 h + 3 of lane half h: after the exchange 2 j + h in place j)
        const auto w01 = __builtin_amdgcn_permlane32_swap(w[0], w[1], false, false);
        const auto w23 = __builtin_amdgcn_permlane32_swap(w[2], w[3], false, false);
        const auto zz = __builtin_amdgcn_permlane32_swap(z[0], z[0], false, false);
        const auto ss = __builtin_amdgcn_permlane32_swap(sb[0], sb[0], false, false);
        const uint32_t w0 = w01[0], w2 = w01[1], w1 = w23[0], w3 = w23[1];
        const uint32_t z0 = zz[0], z1 = zz[1], s0 = ss[0], s1 = ss[1];
        w[0] = w0, w[1] = w1, w[2] = w2, w[3] = w3;
        z[0] = z0, z[1] = z1, sb[0] = s0, sb[1] = s1;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int half = GROUP == 0 ? j / 2 : 0, g = GROUP == 0 ? 2 * b + half : GROUP == 2 ? b / 2 : b;
        const bool first = GROUP == 0 ? j % 2 == 0 : j == 0 && (GROUP == 1 || b % 2 == 0);
        if (j == 2 * half) zb = zero_bias(z[half]);
        if (first) scale[g & 1] = scale_of(sb[half]);
        half2_t d[4];
        decode_pairs(w[j], zb, kc, d);
        const half8_t bf = half8_t{d[0][0], d[0][1], d[1][0], d[1][1], d[2][0], d[2][1], d[3][0], d[3][1]};
#pragma unroll
        for (int a = 0; a < RT; ++a)
          tmp[g & 1][a] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
              af[b & 1][j][a], bf, first ? float16_t(0.0f) : tmp[g & 1][a], 0, 0, 0);
        // With a constant zero as its addend, the compiler may give a matrix
        // instruction a destination that overlaps its operands, which this one
        // (8 passes) writes before it has read them all: they stay alive past it.
        if (first) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int a = 0; a < RT; ++a) asm volatile("" ::"v"(af[b & 1][j][a]), "v"(bf));
        }
        const bool second = GROUP == 0 ? j % 2 == 1 : j == 1 && (GROUP == 1 || b % 2 == 0);
        if (second && g > 0) apply(g - 1, scale[(g - 1) & 1]);
      }
    }
    constexpr int LAST = GROUP == 0 ? 2 * NBLK - 1 : NS - 1;
    apply(LAST, scale[LAST & 1]);
  };

  // stage s has landed once at most the loads of the D - 2 stages after it are
  // in flight; behind the barrier every wave has left the slot that stage
  // s + D - 1 goes into
  Groups gr[D];
  auto step = [&](int s, int c) __attribute__((always_inline)) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(IN_FLIGHT) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    begin(c);
    __builtin_amdgcn_sched_barrier(0);
    load(s + D - 1, (c + D - 1) % D, gr[(c + D - 1) % D]);
    __builtin_amdgcn_sched_barrier(0);
    if (s < s1) compute(c, gr[c]);
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int i = 0; i < D - 1; ++i) load(s0 + i, i, gr[i]);
  __builtin_amdgcn_sched_barrier(0);
  // (whole rounds of D: the words in flight never change registers)
  for (int s = s0; s < s1; s += D) {
#pragma unroll
    for (int c = 0; c < D; ++c) step(s + c, c);
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");  // (the empty loads past the last stage)

  // The sums leave 32 rows at a time through LDS: lane (i, h) holds column i
  // and, in register r, row 8 (r / 4) + 4 h + r % 4.
  float* const stage = reinterpret_cast<float*>(r0);
  const size_t wrow = e * w.N;
  const int chunks = (gated && !part ? COLS / 2 : COLS) / 8;
#pragma unroll
  for (int a = 0; a < RT; ++a) {
    if (32 * a >= t.count) break;
    __builtin_amdgcn_s_barrier();
    float* to = stage + kw * 32 * PITCH + 4 * fh * PITCH + 32 * cw + fi;
#pragma unroll
    for (int r = 0; r < 16; ++r) to[(8 * (r >> 2) + (r & 3)) * PITCH] = acc[a][r];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // eight staged columns of a row, the KW waves' sums added in order
    auto take = [&](int row, int c, float(&v)[8]) __attribute__((always_inline)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float4_t x = *reinterpret_cast<const float4_t*>(&stage[row * PITCH + c + 4 * h]);
#pragma unroll
        for (int q = 1; q < KW; ++q) x += *reinterpret_cast<const float4_t*>(&stage[(q * 32 + row) * PITCH + c + 4 * h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * h + i] = x[i];
      }
    };
#pragma unroll 1
    for (int i = threadIdx.x; i < 32 * chunks; i += WAVES * 64) {
      const int row = i / chunks, c = 8 * (i % chunks);
      const int64_t r = t.row0 + 32 * a + row;
      if (32 * a + row >= t.count) continue;
      float v[8], u[8];
      if (part) {
        // raw sums, part[split][row][N]: the gate's and the up rows' apart
        const int col = n0 + (gated ? 16 * (c >> 5) + (c & 15) : c), n = gated && (c & 16) ? width + col : col;
        if (col >= width) continue;
        take(row, c, v);
        if (p.bias && split == 0)
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] += (float)p.bias[wrow + n + k];
        float* out = part + ((size_t)split * p.R + r) * w.N + n;
        *reinterpret_cast<float4_t*>(out) = *reinterpret_cast<float4_t*>(v);
        *reinterpret_cast<float4_t*>(out + 4) = *reinterpret_cast<float4_t*>(v + 4);
        continue;
      }
      const int n = n0 + c;
      if (n >= width) continue;
      if (gated) {
        const int g = 32 * (c >> 4) + (c & 15);
        take(row, g, v);
        take(row, g + 16, u);
        finish8<true>(v, u, p, wrow, width, r, n, p.activation);
      } else {
        take(row, c, v);
        finish8<false>(v, u, p, wrow, width, r, n, p.activation);
      }
    }
  }
}

template <bool ZP, int GROUP, int XR, int CW, int KW, int D, int SC>
hipError_t launch_stream_as(const PackedArgs& w, const ProductArgs& p, int gs, const StreamPlan& plan, float* part,
                            hipStream_t stream) {
  const int cols = p.gated ? 16 * CW : 32 * CW, width = p.gated ? w.N / 2 : w.N;
  const int tiles_n = (width + cols - 1) / cols;
  const int slots = p.offsets ? row_tiles(p.R, w.E, XR) : (p.R + XR - 1) / XR;
  const int stages = (w.K + SC * KW - 1) / (SC * KW), per = (stages + plan.splits - 1) / plan.splits;
  const auto kernel = w.K % (SC * KW) != 0 ? stream_kernel<ZP, true, GROUP, XR, CW, KW, D, SC>
                                           : stream_kernel<ZP, false, GROUP, XR, CW, KW, D, SC>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(slots * tiles_n), plan.splits), dim3(CW * KW * 64), 0, stream, w, p, gs,
                     tiles_n, per, part);
  return hipGetLastError();
}

template <bool ZP, int GROUP>
hipError_t launch_stream_zg(const PackedArgs& w, const ProductArgs& p, int gs, const StreamPlan& plan, float* part,
                            hipStream_t stream) {
  switch (plan.rows * 100 + plan.cw * 10 + plan.kw) {
    case 1622: return launch_stream_as<ZP, GROUP, 16, 2, 2, 2, 256>(w, p, gs, plan, part, stream);
    case 1624: return launch_stream_as<ZP, GROUP, 16, 2, 4, 2, 256>(w, p, gs, plan, part, stream);
    case 3241: return launch_stream_as<ZP, GROUP, 32, 4, 1, 2, 256>(w, p, gs, plan, part, stream);
    case 3242: return launch_stream_as<ZP, GROUP, 32, 4, 2, 2, 256>(w, p, gs, plan, part, stream);
    case 6441: return launch_stream_as<ZP, GROUP, 64, 4, 1, 3, 128>(w, p, gs, plan, part, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_stream(const PackedArgs& w, const ProductArgs& p, int gshift, const StreamPlan& plan, float* part,
                         hipStream_t stream) {
  if (w.qzeros)
    return gshift == 5   ? launch_stream_zg<true, 0>(w, p, gshift, plan, part, stream)
           : gshift == 6 ? launch_stream_zg<true, 1>(w, p, gshift, plan, part, stream)
                         : launch_stream_zg<true, 2>(w, p, gshift, plan, part, stream);
  return gshift == 5   ? launch_stream_zg<false, 0>(w, p, gshift, plan, part, stream)
         : gshift == 6 ? launch_stream_zg<false, 1>(w, p, gshift, plan, part, stream)
                       : launch_stream_zg<false, 2>(w, p, gshift, plan, part, stream);
}

}  // namespace awq
