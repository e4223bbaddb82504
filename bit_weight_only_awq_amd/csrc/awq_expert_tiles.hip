// Matrix-core bound products (many rows per expert): tiles of up to 128 rows x
// 256 weight rows of X . W'^T with the rows gathered and grouped by expert, and
// the epilogue on the way out.
//
// Mathematics: awq_experts.hip's.  The matrix cores multiply the exact integers
// q - z, and no weight is rounded: a sum over the groups so far is kept as a
// multiple of the last one's scale, and carried to the next one's by the fp32
// ratio of the two before the next group's products are added,
//   A_g = A_{g-1} (s_{g-1} / s_g) + sum_k x_k (q_k - z_g),   sum = A_G s_G
// (Horner's scheme: one multiplication per sum and group, in place, and no
// second set of sums; at most two fp32 roundings per group).  A group of scale
// 0 keeps the multiple and its words are made equal to its zero point.
//
// Bound: the matrix cores at the part's power limit.  Two workgroups per compute
// unit, two waves per SIMD, each wave with all rows of its tile for its 64
// weight rows (32 gate and 32 up rows when gated, so that a lane holds both
// factors of its outputs): every packed word is decoded once per workgroup.
// Rows of X go from HBM into LDS by buffer-to-LDS loads, each lane with its own
// row's offset (a gathered row costs no more than a consecutive one),
// double-buffered; packed words go two steps ahead into registers.  The K loop is
// software-pipelined by hand: the matrix instructions of one 16-channel slice
// run while the next slice's fragments are read from LDS and its words decoded,
// and a tile's rescaling runs beside the matrix instructions of the one before
// it (2048 x 4096 -> 22016 gated: 366-380 us; in a block of its own: 379).
// All 256 registers are in use: 96 rows in groups of 32, which rescale every two
// slices.
//
// One workgroup per tile: its first loads and its epilogue run beside the other
// workgroup of the unit.  Ragged experts: an expert's rows are shared evenly among
// its tiles and the tile's height (in steps of 32 rows) selects a K loop
// unrolled for it, so that a tile multiplies at most 31 rows (63 below 64) that
// do not exist; with more tiles than run at once the tallest come first.
//
// Measured: 2048 x 8192 -> 57344 gated: 1651-1710 us, 1.13-1.17 PFLOP/s (the dense
// library product of the same shape: 1408 us); 2048 x 4096 -> 22016 gated: 363 us,
// in groups of 64: 397, of 32: 513; 1000 tokens x 2 of 8, 4096 -> 22016 gated:
// 402-433 us (264 at the library's rate): whole tiles on two places per unit; 11008
// -> 4096 combined: 242 us with K in 3.  The matrix cores are busy 64%, 48% and 39%
// of their cycles, LDS conflicts 0.3%.  With weights rounded to fp16 (and 256-row
// tiles) they take 1589, 352 (any groups), 430 and 238: exact ones cost 3-5%, 13%
// in groups of 64 and 46% of 32.
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

// A value that is the same in all lanes, in scalar registers (a 64-bit product or
// a division leaves it in vector ones, and every buffer resource made from it
// would be looked up in a loop over the lanes).
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
template <typename T>
__device__ __forceinline__ T* uniform(T* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = uniform((int)(uint32_t)v), hi = uniform((int)(uint32_t)(v >> 32));
  return reinterpret_cast<T*>((uint64_t)hi << 32 | lo);
}

constexpr int kGridX = 1 << 22;  // workgroups of 256 threads along a grid's x: below 2^32 threads
constexpr int kAtOnce = 512;  // workgroups that run at once: two for each of 256 compute units

template <int N>
struct Const {
  static constexpr int value = N;
};

// decode_pairs with its masks in scalar registers: every vector register counts here.
__device__ __forceinline__ void decode_pairs_masks_scalar(uint32_t w, const ZeroBias& b, const DecodeConsts& k,
                                                          half2_t d[4]) {
  auto take = [](uint32_t v, uint32_t mask, uint32_t bias) __attribute__((always_inline)) {
    uint32_t r;
    asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(v), "s"(mask), "v"(bias));
    return as_half2(r);
  };
  const uint32_t w8 = w >> 8;
  d[0] = take(w, k.mask_lo, k.bias_1024) - b.hi;
  d[1] = take(w, k.mask_hi, k.bias_64) - b.lo;
  d[2] = take(w8, k.mask_lo, k.bias_1024) - b.hi;
  d[3] = take(w8, k.mask_hi, k.bias_64) - b.lo;
}

// GROUP: groups of 32 channels (0; K a multiple of 32 only, not of 64), of 64 (1), of 128 and 256 (2).
template <bool ZP, int GROUP, bool GATED>
__global__ __launch_bounds__(256, 2) void tile_kernel(PackedArgs w, ProductArgs p, int gshift, int rows_max,
                                                      int tiles_n, int splits, int steps_per_split,
                                                      float* __restrict__ part) {
  constexpr bool G32 = GROUP == 0;
  constexpr int NB = 2;                     // blocks of 32 weight rows per wave
  constexpr int WN = GATED ? 32 : 64;       // output columns of a wave
  constexpr int MAXT = G32 ? 3 : 4;         // 32-row tiles of the tallest tile
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
  const int block = blockIdx.y * gridDim.x + blockIdx.x;
  if (block >= items) return;
  if (p.offsets != nullptr && items > kAtOnce) row_tiles.tallest_first();

  struct Tile {
    RowTile t;
    int col0, split, s0, s1;  // first output column of the tile; K slice and its steps
  } x;
  // The workgroups that run at once take one contiguous range of items per XCD,
  // tiles in groups of 4 row tiles, so an XCD's L2 sees few row bands and few
  // weight columns at a time.
  {
    const int base = block & ~(kAtOnce - 1);
    const int id = base + xcd_contiguous_tile(block - base, min(kAtOnce, items - base));
    const int group = uniform(id / (4 * tiles_n * splits)), first = group * 4;
    const int gm = min(row_tiles.total - first, 4), in_group = id - group * 4 * tiles_n * splits;
    x.split = uniform(in_group / (gm * tiles_n));
    const int in = in_group - x.split * gm * tiles_n, tn = uniform(in / gm);
    const RowTile t = row_tiles[first + in - tn * gm];
    x.t = RowTile{uniform(t.expert), uniform(t.row0), uniform(t.count)};
    x.col0 = tn * 4 * WN;
    x.s0 = x.split * steps_per_split;
    x.s1 = min(nsteps, x.s0 + steps_per_split);
  }

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
    xbase = uniform(p.rows ? p.x : p.x + x.t.row0 * p.ldx);
    xbytes = uniform(((p.rows ? p.x_rows - 1 : last) * (int)p.ldx + K) * 2);
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
      wbase[b] = uniform(w.qweight + n * (K >> 3));
      wbytes[b] = uniform(rows * (K >> 1));
      rs[b] = make_rsrc(uniform(w.scales + n * G), uniform((rows >> 3) * G * 16));
      rz[b] = make_rsrc(uniform(ZP ? w.qzeros + (n >> 3) * G : w.qweight), ZP ? uniform((rows >> 3) * G * 4) : 0u);
    }
  };
  // One of a step's loads; `buf` is a constant at every call site.  The step
  // goes into the scalar offset, which the range check leaves out: a channel
  // past K is sent out of range by its lane offset, and past the slice's last
  // step the whole buffer is empty (its loads read 0 and cost no traffic).
  auto load_x1 = [&](int step, int s1, int buf, int j) __attribute__((always_inline)) {
    // (K a multiple of 32: the last step's second half)
    const uint32_t off = xoff[j] | (G32 && step * BK + 32 >= K ? xpast : 0u);
    char* const to = (buf ? lx1 : lx0) + 1024 * (wave + 4 * j);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(xbase, step < s1 ? xbytes : 0u),
                                             (__attribute__((address_space(3))) void*)to, 16, off, step * BK * 2, 0, 0);
  };
  struct WRegs {
    u32x4 w[NB];
    uint32_t s[NB], z[NB];
  };
  auto fetch_w = [&](WRegs& r, int step, int s1) __attribute__((always_inline)) {
    const int k0 = step * BK + 32 * fh;
    const uint32_t past = G32 && k0 >= K ? kOutOfRange : 0u;
    const int grp = k0 >> gshift;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const __amdgpu_buffer_rsrc_t rw = make_rsrc(wbase[b], step < s1 ? wbytes[b] : 0u);
      r.w[b] = __builtin_bit_cast(u32x4,
                                  __builtin_amdgcn_raw_buffer_load_b128(rw, woff | past, step * (BK / 2), 0));
      r.s[b] = __builtin_amdgcn_raw_buffer_load_b16(rs[b], (soff + grp * 16) | past, 0, 0);
      r.z[b] = ZP ? __builtin_amdgcn_raw_buffer_load_b32(rz[b], (zoff + grp * 4) | past, 0, 0) : 0u;
    }
  };

  WRegs w0, w1;
  setup(x);
#pragma unroll
  for (int j = 0; j < MAXT; ++j)
    if (j <= xlast) load_x1(x.s0, x.s1, 0, j);
  fetch_w(w0, x.s0, x.s1);
  fetch_w(w1, x.s0 + 1, x.s1);

  const int fsw = (fi >> 1) & 7;
  // the K loop of a tile of WMT 32-row tiles, its first loads landed
  auto multiply = [&](auto wmt, auto& acc, const Tile& x) __attribute__((always_inline)) {
    constexpr int WMT = decltype(wmt)::value;
    ZeroBias zb[NB];
    float unit[NB];  // what the sums are multiples of
    half8_t af[2][WMT], bf[2][NB];
    auto load_x = [&](int step, int buf) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < WMT; ++j) load_x1(step, x.s1, buf, j);
    };
    auto scale_of = [&](uint32_t bits) __attribute__((always_inline)) {
      return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
    };
    // A step's zero points and scales, its words where a scale is zero (they
    // become their zero point, so that the group adds nothing); for groups of 32
    // the lane halves exchange words, so that a slice lies in one group.
    auto prep = [&](WRegs& r) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t z[2] = {ZP ? (r.z[b] >> zshift) & 15u : 8u, 0u}, sb[2] = {r.s[b], 0u};
        if (__ballot((uint16_t)(sb[0] << 1) == 0) != 0) {
          const bool none = (uint16_t)(sb[0] << 1) == 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) r.w[b][i] = none ? z[0] * 0x11111111u : r.w[b][i];
        }
        if constexpr (G32) {
          // (words 4 h .. 4 h + 3 of lane half h: after the exchange 2 i + h in slice i)
          const auto w01 = __builtin_amdgcn_permlane32_swap(r.w[b][0], r.w[b][1], false, false);
          const auto w23 = __builtin_amdgcn_permlane32_swap(r.w[b][2], r.w[b][3], false, false);
          const uint32_t a0 = w01[0], a2 = w01[1], a1 = w23[0], a3 = w23[1];
          r.w[b] = u32x4{a0, a1, a2, a3};
          const auto zz = __builtin_amdgcn_permlane32_swap(z[0], z[0], false, false);
          const auto ss = __builtin_amdgcn_permlane32_swap(sb[0], sb[0], false, false);
          const uint32_t z0 = zz[0], z1 = zz[1], t0 = ss[0], t1 = ss[1];
          z[0] = z0, z[1] = z1, sb[0] = t0, sb[1] = t1;
        }
        zb[b] = zero_bias(z[0]);
        r.z[b] = z[1];
        r.s[b] = sb[0] | sb[1] << 16;
      }
    };
    // From multiples of the group before's scale to multiples of this one's.
    auto ratios = [&](const WRegs& r, int g, float (&ratio)[NB]) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float s = scale_of(g ? r.s[b] >> 16 : r.s[b]);
        const float to = s == 0.0f ? unit[b] : s;
        ratio[b] = unit[b] / to;
        unit[b] = to;
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // slice ks: channels 32 h + 8 ks + j of lane half h's 32 (groups of 32: 16 ks +
    // 8 h + j), for X and W alike
    auto read_a = [&](int buf, int ks, int d) __attribute__((always_inline)) {
      const char* xa = (buf ? lx1 : lx0) + fi * 128 + 16 * ((G32 ? 2 * ks + fh : 4 * fh + ks) ^ fsw);
#pragma unroll
      for (int a = 0; a < WMT; ++a) af[d][a] = *reinterpret_cast<const half8_t*>(xa + 32 * 128 * a);
    };
    auto decode_b = [&](const WRegs& r, int ks, int d) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        half2_t p[4];
        decode_pairs_masks_scalar(r.w[b][ks], zb[b], kc, p);
        bf[d][b] = half8_t{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
      }
    };
    auto mfmas = [&](int d, const float* ratio) __attribute__((always_inline)) {
#pragma unroll
      for (int a = 0; a < WMT; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (ratio != nullptr) acc[a][b] *= ratio[b];
          acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[d][a], bf[d][b], acc[a][b], 0, 0, 0);
        }
    };
    // per 32-row tile: one LDS read, one MFMA, three VALU, the other MFMA, one VALU;
    // rescaling, 16 multiplications before each MFMA
    auto interleave = [&](bool rescaled) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < WMT; ++i) {
        if (rescaled) {
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 18, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 18, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          continue;
        }
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 1, 0);
      }
    };
    // one step with its tile in buffer c and its words in wc (wnx: the next
    // step's).  On entry af[0] / bf[0] hold slice 0, on exit the next step's.
    auto body = [&](int c, WRegs& wc, WRegs& wnx, int step, bool hand) __attribute__((always_inline)) {
      float ratio[NB];
#pragma unroll
      for (int ks = 0; ks < 3; ++ks) {
        const int d = ks & 1;
        // (groups of 128: slices of K begin at even steps; of 256: with ratios of 1 in the middle)
        const bool first = ks == 0 ? GROUP != 2 || c == 0 : G32 && ks == 2;
        if (first) ratios(wc, ks / 2, ratio);
        if (G32 && ks == 1)
#pragma unroll
          for (int b = 0; b < NB; ++b) zb[b] = zero_bias(wc.z[b]);
        read_a(c, ks + 1, d ^ 1);
        decode_b(wc, ks + 1, d ^ 1);
        if (ks == 2) fetch_w(wc, step + 2, x.s1);
        mfmas(d, first ? ratio : nullptr);
        interleave(first);
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
      mfmas(1, nullptr);
      interleave(false);
      __builtin_amdgcn_sched_barrier(0);
    };
    float zero = 0.0f;
    asm volatile("" : "+v"(zero));  // (a constant would be kept as a tuple of registers, or spilled as one)
#pragma unroll
    for (int a = 0; a < WMT; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[a][b] = float16_t(zero);
#pragma unroll
    for (int b = 0; b < NB; ++b) unit[b] = 1.0f;
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
#pragma unroll
    for (int a = 0; a < WMT; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[a][b][r] *= unit[b];
  };

  // The sums leave 32 rows at a time through LDS, so that a thread finishes 8
  // consecutive columns of a row with 128-bit loads and stores; one copy of the
  // code serves all 32-row tiles (unrolled over the accumulators it outgrew the
  // instruction cache).
  auto finish = [&](auto wmt, auto& acc, const Tile& x) __attribute__((always_inline)) {
    constexpr int WMT = decltype(wmt)::value;
    constexpr int COLS = 4 * 32 * NB, CHUNKS = 4 * WN / 8;  // staged columns; 8-column chunks of a row's outputs
    const size_t wrow = (size_t)x.t.expert * w.N;
#pragma unroll 1
    for (int cur = 0; 32 * cur < x.t.count; ++cur) {
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
  };

  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the first step's loads
  lds_barrier();
  // (the accumulators live within one case: no registers to match between
  // the K loops of different heights)
  auto tile = [&](auto wmt) __attribute__((always_inline)) {
    float16_t acc[decltype(wmt)::value][NB];
    multiply(wmt, acc, x);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // (the empty loads past the last step)
    finish(wmt, acc, x);
  };
  switch ((x.t.count + 31) >> 5) {
    case 1:
    case 2: tile(Const<2>{}); break;
    case 3: tile(Const<3>{}); break;
    default:
      if constexpr (MAXT > 3) tile(Const<MAXT>{});
  }
}

template <bool ZP, int GROUP>
hipError_t launch_tiles_zk(const PackedArgs& w, const ProductArgs& p, int gs, const TilePlan& plan, float* part,
                           hipStream_t stream) {
  const int width = p.gated ? w.N / 2 : w.N, tbn = p.gated ? 128 : 256;
  const int tiles_n = (width + tbn - 1) / tbn;
  const int slots = p.offsets ? row_tiles(p.R, w.E, plan.rows) : (p.R + plan.rows - 1) / plan.rows;
  const int64_t items = (int64_t)slots * tiles_n * plan.splits;
  const auto kernel = p.gated ? tile_kernel<ZP, GROUP, true> : tile_kernel<ZP, GROUP, false>;
  const int64_t x = items < kGridX ? items : kGridX;  // (a multiple of kAtOnce, or one row of the grid)
  hipLaunchKernelGGL(kernel, dim3((unsigned)x, (unsigned)((items + x - 1) / x)), dim3(256), 0, stream,
                     w, p, gs, plan.rows, tiles_n, plan.splits, plan.steps_per_split, part);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_tiles(const PackedArgs& w, const ProductArgs& p, int gshift, const TilePlan& plan, float* part,
                        hipStream_t stream) {
  // no group of 128 is cut, and a tile has the kernel's rows at most
  if ((plan.splits > 1 && (plan.steps_per_split & 1)) || plan.rows > (gshift == 5 ? 96 : 128)) return hipErrorInvalidValue;
  const int group = gshift == 5 ? 0 : gshift == 6 ? 1 : 2;
  if (w.qzeros)
    return group == 0   ? launch_tiles_zk<true, 0>(w, p, gshift, plan, part, stream)
           : group == 1 ? launch_tiles_zk<true, 1>(w, p, gshift, plan, part, stream)
                        : launch_tiles_zk<true, 2>(w, p, gshift, plan, part, stream);
  return group == 0   ? launch_tiles_zk<false, 0>(w, p, gshift, plan, part, stream)
         : group == 1 ? launch_tiles_zk<false, 1>(w, p, gshift, plan, part, stream)
                      : launch_tiles_zk<false, 2>(w, p, gshift, plan, part, stream);
}

}  // namespace awq
