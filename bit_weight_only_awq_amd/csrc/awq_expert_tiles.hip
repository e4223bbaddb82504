// Matrix-core bound products (many rows per expert): tiles of up to 256 rows x
// 256 weight rows of X . W'^T with the rows gathered and grouped by expert, and
// the epilogue on the way out.
//
// Mathematics: awq_experts.hip's, with W' = fp16((q - z) s), one rounding per
// weight (relative 2^-11; products exact, sums fp32), which is what lets one
// decoded fragment feed all row tiles of a wave.
//
// Bound: the matrix cores at the part's power limit.  One wave per SIMD, each
// holding all rows of the tile for its 64 weight rows (32 gate and 32 up rows
// when gated, so that a lane holds both factors of its outputs): every packed
// word is decoded once per workgroup.  Rows of X go from HBM into LDS by
// buffer-to-LDS loads, each lane with its own row's offset (a gathered row
// costs no more than a consecutive one), double-buffered; packed words go two
// steps ahead into registers.  The K loop is software-pipelined by hand, as a
// single wave per SIMD has no other to hide latency behind: the matrix
// instructions of one 16-channel slice run while the next slice's fragments
// are read from LDS and its words decoded.
//
// The workgroups are persistent, one per compute unit, each taking every
// gridDim-th tile: a tile's first loads are issued before the epilogue of the
// tile before it, and its output is written while the next one multiplies.
// Ragged experts: an expert's rows are shared evenly among its tiles and the
// tile's height (in steps of 32 rows) selects a K loop unrolled for it, so that
// a tile multiplies at most 31 rows (63 below 128) that do not exist.
//
// Measured: 2048 x 8192 -> 57344 gated: 1570 us, 1.23 PFLOP/s (the dense library
// product of the same shape: 1408 us); 1000 tokens x 2 of 8, 4096 -> 22016 gated:
// 416 us (264 at that rate): whole rounds of tiles and ragged heights; 11008 ->
// 4096 of the same rows: 232 us, one round of 160-176 tiles on 256 compute units.
// The matrix cores are busy 63% of the gated tiles' cycles, LDS conflicts 0.3%.
#include "awq_epilogue.hpp"
#include "awq_launch_fused.hpp"

namespace awq {
namespace {

constexpr int BK = 64;  // channels per step
constexpr uint32_t kOutOfRange = 0x80000000u;  // a buffer offset past every resource: loads return 0

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

// Chunk of 16 bytes c of row r of an LDS tile sits in slot c ^ ((r >> 1) & 7):
// the fragment reads (16 consecutive rows at one chunk) touch every bank once.
__device__ __forceinline__ int swz_chunk(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }

// A workgroup barrier that orders LDS accesses only: global loads and stores
// stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

int compute_units() {
  static const int units = [] {
    int dev = 0, n = 0;
    return hipGetDevice(&dev) == hipSuccess &&
                   hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && n > 0
               ? n
               : 256;
  }();
  return units;
}

template <int N>
struct Const {
  static constexpr int value = N;
};

template <bool ZP, bool KTAIL, bool GATED>
__global__ __launch_bounds__(256) void tile_kernel(PackedArgs w, ProductArgs p, int gshift, int rows_max, int tiles_n,
                                                   int splits, int steps_per_split, float* __restrict__ part) {
  constexpr int NB = 2;                     // blocks of 32 weight rows per wave
  constexpr int WN = GATED ? 32 : 64;       // output columns of a wave
  constexpr int MAXT = 8;                   // 32-row tiles of the tallest tile
  constexpr int W_LOADS = NB * (ZP ? 3 : 2);  // vector loads of one step's weights
  // two arrays, so that the wait for buffer-to-LDS loads before an LDS read
  // covers only the loads into the array being read
  __shared__ __attribute__((aligned(1024))) char lx0[MAXT * 32 * BK * 2], lx1[MAXT * 32 * BK * 2];
  // 32 rows of sums on their way out; the pitch puts the two lane halves' rows
  // (4 apart) in the two halves of the banks
  constexpr int PITCH = 128 * NB + 8;
  __shared__ __attribute__((aligned(16))) float stage[32 * PITCH];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fi = lane & 31, fh = lane >> 5;
  const int K = w.K, width = GATED ? w.N >> 1 : w.N, G = K >> gshift;
  const int nsteps = (K + BK - 1) / BK;
  const DecodeConsts kc;
  RowTiles row_tiles(p.offsets, w.E, p.R, rows_max, 32);
  const int items = row_tiles.total * tiles_n * splits;
  const bool rounds = p.offsets != nullptr && items > (int)gridDim.x;
  if (rounds) row_tiles.tallest_first();

  struct Tile {
    RowTile t;
    int col0, split, s0, s1;  // first output column of the tile; K slice and its steps
  };
  // This workgroup's item of a round.  The items of a round (one per workgroup)
  // lie in one contiguous range per XCD, tiles in groups of 4 row tiles, so an
  // XCD's L2 sees few row bands and few weight columns at a time.  The
  // rounds of ragged experts begin with the tallest tiles and every other one goes
  // backwards, so that the workgroups' shares come out alike (1000 tokens x 2 of
  // 8, 4096 -> 28672 gated: 533 us, 557 in the experts' order).
  auto locate = [&](int round, Tile& x) __attribute__((always_inline)) {
    const int base = round * (int)gridDim.x, here = min((int)gridDim.x, items - base);
    int at;
    if (rounds) {
      at = xcd_contiguous_tile(blockIdx.x, gridDim.x);
      if (round & 1) at = gridDim.x - 1 - at;
    } else {
      at = (int)blockIdx.x < here ? xcd_contiguous_tile(blockIdx.x, here) : here;
    }
    if (at >= here) return false;
    const int id = base + at, group = id / (4 * tiles_n * splits), first = group * 4;
    const int gm = min(row_tiles.total - first, 4), in_group = id - group * 4 * tiles_n * splits;
    x.split = in_group / (gm * tiles_n);
    const int in = in_group - x.split * gm * tiles_n, tn = in / gm;
    x.t = row_tiles[first + in - tn * gm];
    x.col0 = tn * 4 * WN;
    x.s0 = x.split * steps_per_split;
    x.s1 = min(nsteps, x.s0 + steps_per_split);
    return true;
  };

  // X: the 8-row groups of the tile go to the waves in turn, group wave + 4 j to
  // wave `wave`'s j-th load of a step (rows past the tile's: its last row, never stored)
  const void *xbase, *wbase[NB];
  uint32_t xbytes, wbytes[NB];
  __amdgpu_buffer_rsrc_t rs[NB], rz[NB];
  uint32_t xoff[MAXT];
  int xlast = 0;  // 32-row tiles - 1
  const int xrow = 8 * wave + (lane >> 3), xchunk = swz_chunk(xrow, lane & 7);  // 32 j more rows: the same chunk
  const uint32_t xpast = xchunk >= 4 ? kOutOfRange : 0u;
  // W: lane (i, h) = (lane % 32, lane / 32) of this wave holds row i of each of
  // its NB blocks of 32 weight rows; rows past N lie past the resources and read as 0
  const uint32_t woff = (uint32_t)fi * (K >> 1) + fh * 16;
  const uint32_t soff = (uint32_t)(((fi >> 3) * G * 8 + (fi & 7)) * 2), zoff = (uint32_t)((fi >> 3) * G * 4);
  const int zshift = 4 * (fi & 7);
  auto setup = [&](const Tile& x) __attribute__((always_inline)) {
    const int last = x.t.count - 1;
    xlast = last >> 5;
    xbase = p.rows ? p.x : p.x + x.t.row0 * p.ldx;
    xbytes = (uint32_t)((p.rows ? p.x_rows - 1 : last) * (int)p.ldx + K) * 2;
#pragma unroll
    for (int j = 0; j < MAXT; ++j) {
      int r = min(xrow + 32 * j, last);
      if (p.rows) r = min(max(p.rows[x.t.row0 + r] / p.slots_per_row, 0), p.x_rows - 1);
      xoff[j] = (uint32_t)(r * (int)p.ldx + xchunk * 8) * 2;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int col = x.col0 + wave * WN + (GATED ? 0 : 32 * b);    // first output column
      const int rows = min(max(width - col, 0), 32);                // a multiple of 8
      const size_t n = (size_t)x.t.expert * w.N + (GATED ? b * width : 0) + min(col, width - 8);
      wbase[b] = w.qweight + n * (K >> 3);
      wbytes[b] = (uint32_t)rows * (K >> 1);
      rs[b] = make_rsrc(w.scales + n * G, (uint32_t)(rows >> 3) * G * 16);
      rz[b] = make_rsrc(ZP ? w.qzeros + (n >> 3) * G : w.qweight, ZP ? (uint32_t)(rows >> 3) * G * 4 : 0u);
    }
  };
  // One of a step's loads; `buf` is a constant at every call site.  The step
  // goes into the scalar offset, which the range check leaves out: a channel
  // past K is sent out of range by its lane offset, and past the slice's last
  // step the whole buffer is empty (its loads read 0 and cost no traffic).
  auto load_x1 = [&](int step, int s1, int buf, int j) __attribute__((always_inline)) {
    // (K a multiple of 32: the last step's second half)
    const uint32_t off = xoff[j] | (KTAIL && step == nsteps - 1 ? xpast : 0u);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        make_rsrc(xbase, step < s1 ? xbytes : 0u), (__attribute__((address_space(3))) void*)((buf ? lx1 : lx0) + 1024 * (wave + 4 * j)), 16, off, step * BK * 2,
        0, 0);
  };
  struct WRegs {
    u32x4 w[NB];
    uint32_t s[NB], z[NB];
  };
  auto fetch_w = [&](WRegs& r, int step, int s1) __attribute__((always_inline)) {
    const int k0 = step * BK + 32 * fh;
    const int grp = k0 >> gshift;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      r.w[b] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                             make_rsrc(wbase[b], step < s1 ? wbytes[b] : 0u), woff | (KTAIL && k0 >= K ? kOutOfRange : 0u), step * (BK / 2), 0));
      r.s[b] = __builtin_amdgcn_raw_buffer_load_b16(rs[b], soff + grp * 16, 0, 0);
      r.z[b] = ZP ? __builtin_amdgcn_raw_buffer_load_b32(rz[b], zoff + grp * 4, 0, 0) : 0u;
    }
  };

  WRegs w0, w1;
  // the first loads of a tile
  auto begin = [&](const Tile& x) __attribute__((always_inline)) {
    setup(x);
#pragma unroll
    for (int j = 0; j < MAXT; ++j)
      if (j <= xlast) load_x1(x.s0, x.s1, 0, j);
    fetch_w(w0, x.s0, x.s1);
    fetch_w(w1, x.s0 + 1, x.s1);
  };

  const int fsw = (fi >> 1) & 7;
  // the K loop of a tile of WMT 32-row tiles, its first loads landed
  auto multiply = [&](auto wmt, auto& acc, const Tile& x) __attribute__((always_inline)) {
    constexpr int WMT = decltype(wmt)::value;
    ZeroBias zb[NB];
    half2_t s2[NB];
    half8_t af[2][WMT], bf[2][NB];
    auto load_x = [&](int step, int buf) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < WMT; ++j) load_x1(step, x.s1, buf, j);
    };
    auto prep = [&](const WRegs& r) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        zb[b] = zero_bias(ZP ? ((r.z[b] >> zshift) & 15u) : 8u);
        s2[b] = splat2(__builtin_bit_cast(_Float16, (uint16_t)r.s[b]));
      }
    };
    // slice ks: channels 32 h + 8 ks + j of lane half h's 32, for X and W alike
    auto read_a = [&](int buf, int ks, int d) __attribute__((always_inline)) {
      const char* xa = (buf ? lx1 : lx0) + fi * 128 + 16 * ((4 * fh + ks) ^ fsw);
#pragma unroll
      for (int a = 0; a < WMT; ++a) af[d][a] = *reinterpret_cast<const half8_t*>(xa + 32 * 128 * a);
    };
    auto decode_b = [&](const WRegs& r, int ks, int d) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < NB; ++b) bf[d][b] = decode_word_scaled(r.w[b][ks], zb[b], kc, s2[b]);
    };
    auto mfmas = [&](int d) __attribute__((always_inline)) {
#pragma unroll
      for (int a = 0; a < WMT; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[d][a], bf[d][b], acc[a][b], 0, 0, 0);
    };
    // per 32-row tile: one LDS read, one MFMA, three VALU, the other MFMA, one VALU
    auto interleave = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < WMT; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 1, 0);
      }
    };
    // one step with its tile in buffer c and its words in wc (wnx: the next
    // step's).  On entry af[0] / bf[0] hold slice 0, on exit the next step's.
    auto body = [&](int c, WRegs& wc, const WRegs& wnx, int step, bool hand) __attribute__((always_inline)) {
#pragma unroll
      for (int ks = 0; ks < 3; ++ks) {
        const int d = ks & 1;
        read_a(c, ks + 1, d ^ 1);
        decode_b(wc, ks + 1, d ^ 1);
        if (ks == 2) fetch_w(wc, step + 2, x.s1);
        mfmas(d);
        interleave();
        __builtin_amdgcn_sched_barrier(0);
      }
      if (hand) {
        // the next tile has landed (only this step's weight loads are younger),
        // and no wave still reads this one
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(W_LOADS) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        load_x(step + 2, c);
        prep(wnx);
        read_a(c ^ 1, 0, 0);
        decode_b(wnx, 0, 0);
      }
      mfmas(1);
      interleave();
      __builtin_amdgcn_sched_barrier(0);
    };
    float zero = 0.0f;
    asm volatile("" : "+v"(zero));  // (a constant would be kept as a tuple of registers, or spilled as one)
#pragma unroll
    for (int a = 0; a < WMT; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[a][b] = float16_t(zero);
    load_x(x.s0 + 1, 1);
    prep(w0);
    read_a(0, 0, 0);
    decode_b(w0, 0, 0);
    int step = x.s0;
    for (; step + 1 < x.s1; step += 2) {
      body(0, w0, w1, step, true);
      body(1, w1, w0, step + 1, true);
    }
    if (step < x.s1) body(0, w0, w1, step, false);
  };

  // The sums leave 32 rows at a time
  // through LDS, so that a thread finishes 8 consecutive columns of a row with
  // 128-bit loads and stores; one copy of the code serves all 32-row tiles
  // (unrolled over the accumulators it outgrew the instruction cache).
  // Between the first and the second of them the next tile's first loads are
  // waited for, ahead of the bulk of the stores that would be waited for with them.
  auto finish = [&](auto wmt, auto& acc, const Tile& x) __attribute__((always_inline)) {
    constexpr int WMT = decltype(wmt)::value;
    constexpr int COLS = 4 * 32 * NB, CHUNKS = 4 * WN / 8;  // staged columns; 8-column chunks of a row's outputs
    const size_t wrow = (size_t)x.t.expert * w.N;
#pragma unroll 1
    for (int cur = 0; 32 * cur < x.t.count; ++cur) {
      if (cur == 1) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      lds_barrier();
      // 32-row tile `cur` to LDS: lane (i, h) holds column i of each block and,
      // in register r, row 8 (r / 4) + 4 h + r % 4
#pragma unroll
      for (int a = 0; a < WMT; ++a)
        if (a == cur) {
          // (keeps the compiler from merging the cases into one load through a
          // pointer, which would put the accumulators in memory)
          asm volatile("" ::: "memory");
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r)
              stage[(8 * (r >> 2) + 4 * fh + (r & 3)) * PITCH + (GATED ? 128 * b + 32 * wave : 64 * wave + 32 * b) +
                    fi] = acc[a][b][r];
        }
      lds_barrier();
#pragma unroll 1
      for (int i = threadIdx.x; i < 32 * (part ? COLS / 8 : CHUNKS); i += 256) {
        if (part) {
          // raw sums, part[split][row][N]: the gate's and the up rows' apart
          const int row = i / (COLS / 8), c = 8 * (i % (COLS / 8));
          const int col = x.col0 + (GATED ? c & 127 : c), n = GATED && c >= 128 ? width + col : col;
          if (32 * cur + row >= x.t.count || col >= width) continue;
          float* to = part + ((size_t)x.split * p.R + x.t.row0 + 32 * cur + row) * w.N + n;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float4_t v = *reinterpret_cast<const float4_t*>(&stage[row * PITCH + c + 4 * h]);
            if (p.bias && x.split == 0)
#pragma unroll
              for (int k = 0; k < 4; ++k) v[k] += (float)p.bias[wrow + n + 4 * h + k];
            *reinterpret_cast<float4_t*>(to + 4 * h) = v;
          }
          continue;
        }
        const int row = i / CHUNKS, c = 8 * (i % CHUNKS), n = x.col0 + c;
        const int64_t r = x.t.row0 + 32 * cur + row;
        if (32 * cur + row >= x.t.count || n >= width) continue;
        float v[8], u[8];
        *reinterpret_cast<float4_t*>(v) = *reinterpret_cast<const float4_t*>(&stage[row * PITCH + c]);
        *reinterpret_cast<float4_t*>(v + 4) = *reinterpret_cast<const float4_t*>(&stage[row * PITCH + c + 4]);
        if constexpr (GATED) {
          *reinterpret_cast<float4_t*>(u) = *reinterpret_cast<const float4_t*>(&stage[row * PITCH + 128 + c]);
          *reinterpret_cast<float4_t*>(u + 4) = *reinterpret_cast<const float4_t*>(&stage[row * PITCH + 132 + c]);
        }
        finish8<GATED>(v, u, p, wrow, width, r, n, p.activation);
      }
    }
    if (x.t.count <= 32) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier();
  };

  Tile x, next;
  if (!locate(0, x)) return;
  begin(x);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  lds_barrier();
  int round = 1;
  bool more;
  // (the accumulators live within one case: no registers to match between
  // the K loops of different heights)
  auto tile = [&](auto wmt) __attribute__((always_inline)) {
    float16_t acc[decltype(wmt)::value][NB];
    multiply(wmt, acc, x);
    more = locate(round, next);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // (the empty loads past the last step)
    lds_barrier();                                    // no wave still reads the tile
    if (more) begin(next);
    finish(wmt, acc, x);
  };
  do {
    switch ((x.t.count + 31) >> 5) {
      case 1:
      case 2: tile(Const<2>{}); break;
      case 3:
      case 4: tile(Const<4>{}); break;
      case 5: tile(Const<5>{}); break;
      case 6: tile(Const<6>{}); break;
      case 7: tile(Const<7>{}); break;
      default: tile(Const<8>{}); break;
    }
    x = next;
    ++round;
  } while (more);
}

template <bool ZP, bool KTAIL>
hipError_t launch_tiles_zk(const PackedArgs& w, const ProductArgs& p, int gs, const TilePlan& plan, float* part,
                           hipStream_t stream) {
  const int width = p.gated ? w.N / 2 : w.N, tbn = p.gated ? 128 : 256;
  const int tiles_n = (width + tbn - 1) / tbn;
  const int slots = p.offsets ? row_tiles(p.R, w.E, plan.rows) : (p.R + plan.rows - 1) / plan.rows;
  const int64_t items = (int64_t)slots * tiles_n * plan.splits;
  const auto kernel = p.gated ? tile_kernel<ZP, KTAIL, true> : tile_kernel<ZP, KTAIL, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(items < compute_units() ? items : compute_units())), dim3(256), 0, stream,
                     w, p, gs, plan.rows, tiles_n, plan.splits, plan.steps_per_split, part);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_tiles(const PackedArgs& w, const ProductArgs& p, int gshift, const TilePlan& plan, float* part,
                        hipStream_t stream) {
  const bool tail = w.K % BK != 0;
  if (w.qzeros)
    return tail ? launch_tiles_zk<true, true>(w, p, gshift, plan, part, stream)
                : launch_tiles_zk<true, false>(w, p, gshift, plan, part, stream);
  return tail ? launch_tiles_zk<false, true>(w, p, gshift, plan, part, stream)
              : launch_tiles_zk<false, false>(w, p, gshift, plan, part, stream);
}

}  // namespace awq
