// Shared by the attention kernels: 32 rows of queries against 32 keys on the
// matrix cores.
//
// Mathematics: a wave keeps, for each of its 32 rows, the running maximum m of the
// scores, the sum l of the weights 2^((score - m) c) with c = scale log2(e), and
// the weighted sum of the values, one pass over the keys.  Scores are formed
// transposed, keys x queries, so that a lane holds 16 scores of one row (lane %
// 32) and its partner 32 lanes away the other 16: maximum and sum need one
// exchange, and a change of the maximum scales a lane's sums by a number it
// has.  The weights, rounded to fp16 (relative 2^-11, as the values are), are then in
// place as the second operand of the product with the values, whose first operand
// comes out of LDS transposed; both follow the same order of keys (lane half h holds
// keys 8 j + 4 h .. + 3), so nothing is exchanged.  Sums are fp32.
//
// The maximum lags: sums are rescaled only once a score passes it by a factor of
// 2^8, which fp16 holds for weights and fp32 for sums.
#pragma once

#include <type_traits>

#include "awq_cache.hpp"

namespace awq {

typedef short short4_t __attribute__((ext_vector_type(4)));
// (Addresses in LDS stay in its own address space: as general ones they would lose which array they point into, and
// with that the compiler's knowledge that a read and a load into another stage do not meet.)
#define AWQ_LDS __attribute__((address_space(3)))
typedef AWQ_LDS char lds_char;

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLag = 8.0f;  // the maximum lags by at most this power of two

// Rows of D halves in LDS, as 16-byte chunks: chunk c of row r is at chunk c ^ swizzle(r), so that what
// one instruction reads lies in different banks (16 rows of one chunk for keys, 4 rows of 4 chunks for values).
template <int D>
struct Tile {
  static constexpr int CHUNKS = D / 8, ROW = D * 2;
  static constexpr int LOADS = D / 32;  // loads of 64 chunks per 16 rows
  static __device__ __forceinline__ int key_swizzle(int r) {
    return D == 64 ? (r >> 1) & 7 : D == 96 ? (r >> 2) & 3 : r & 15;
  }
  static __device__ __forceinline__ int value_swizzle(int r) {
    return D == 64 ? ((r >> 1) & 1) << 2 : D == 96 ? 0 : (r & 3) << 2;
  }
};

// Where a lane reads from, in bytes from the first of 16 rows, for each of the loads of 64 chunks that bring them:
// the chunks' swizzles are powers of two apart from load to load (but not of rows of 12 chunks).
template <int D>
struct Sources {
  using T = Tile<D>;
  static constexpr int KEPT = D == 96 ? 3 : 1, ROWS = 64 / T::CHUNKS;
  uint32_t keys[KEPT], values[KEPT];
  // loads `first`, `first` + 1, ... (a multiple of 4)
  __device__ __forceinline__ Sources(int lane, int first) {
#pragma unroll
    for (int i = 0; i < KEPT; ++i) {
      const int at = 64 * (first + i) + lane, r = at / T::CHUNKS, c = at % T::CHUNKS;
      keys[i] = (uint32_t)(r * T::ROW + 16 * (c ^ T::key_swizzle(r)));
      values[i] = (uint32_t)(r * T::ROW + 16 * (c ^ T::value_swizzle(r)));
    }
  }
  __device__ __forceinline__ uint32_t key(int i) const {
    return D == 96 ? keys[i] : (keys[0] ^ (uint32_t)(16 * (D == 64 ? 4 * i : ROWS * i))) + 1024 * i;
  }
  __device__ __forceinline__ uint32_t value(int i) const {
    return D == 96 ? values[i] : (values[0] ^ (uint32_t)(D == 256 ? 128 * (i & 1) : 0)) + 1024 * i;
  }
};

// 16 bytes per lane from `from` (a byte address per lane) into LDS, lane after lane.
__device__ __forceinline__ void load_to_lds(const char* from, lds_char* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (AWQ_LDS void*)to, 16, 0, 0);
}

__device__ __forceinline__ float both_halves_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false,
                                                  false);
  const uint32_t r0 = r[0], r1 = r[1];
  return fmaxf(__builtin_bit_cast(float, r0), __builtin_bit_cast(float, r1));
}
__device__ __forceinline__ float both_halves_sum(float v) { return swap_sum32(v, v); }

// What 32 rows have gathered: sums[b][i] is channel 32 b + 8 (i / 4) + 4 (lane /
// 32) + i % 4 of row lane % 32; `sum` is the lane's share of l.
template <int D>
struct Gathered {
  float16_t sums[D / 32];
  float top, sum;
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int b = 0; b < D / 32; ++b) sums[b] = float16_t(0.0f);
    top = -INFINITY;
    sum = 0.0f;
  }
};

// Fragments of 32 rows' queries: row lane % 32, channels 16 j + 8 (lane / 32) .. + 7.  Where a head is 256 wide they
// are in LDS, a wave's 64 times 16 bytes for each j (in registers with everything else, they would not all fit).
template <int D>
struct Queries {
  static constexpr int BYTES = 0;  // of LDS, for a wave
  half8_t part[D / 16];
  __device__ __forceinline__ void place(lds_char*) {}
  __device__ __forceinline__ void put(int j, half8_t v) { part[j] = v; }
};
template <>
struct Queries<256> {
  static constexpr int BYTES = 16 * 1024;
  lds_char* at;
  __device__ __forceinline__ void place(lds_char* to) { at = to + 16 * __lane_id(); }
  __device__ __forceinline__ void put(int j, half8_t v) { *(AWQ_LDS half8_t*)(at + 1024 * j) = v; }
};

// Which of a block's keys the rows see: those of each 16 up to `limit` (the row's own place, less that of the first
// of them); `all`: all rows see all 32.
struct Seen {
  int limit0, limit1;
  bool all;
};

__device__ __forceinline__ bool finite16(uint32_t h) { return (h & 0x7C00u) != 0x7C00u; }

// Values that some row must not see, not as 0 times infinity either: of ROWS rows at LDS address `values`, those
// behind `least` (of their 16) that are not finite become 0, and where a row of the tile does see them (up to `most`),
// the row's bit is returned: the product below gives these one by one.  `threads` threads, `id` this one's number;
// each returns what it met.
template <int D, int ROWS, typename Bound>
__device__ __forceinline__ uint64_t hide_strange(lds_char* values, int id, int threads, Bound bound) {
  using T = Tile<D>;
  uint64_t met = 0;
#pragma unroll 1
  for (int i = id; i < ROWS * T::CHUNKS; i += threads) {
    const int row = i / T::CHUNKS;
    int least, most;
    bound(row >> 4, least, most);
    if ((row & 15) <= least) continue;
    AWQ_LDS u32x4* at = (AWQ_LDS u32x4*)(values + 16 * i);
    u32x4 v = *at;
    bool bad = false;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (!finite16(v[w])) bad = true, v[w] &= 0xFFFF0000u;
      if (!finite16(v[w] >> 16)) bad = true, v[w] &= 0x0000FFFFu;
    }
    if (!bad) continue;
    *at = v;
    if ((row & 15) <= most) met |= 1ull << row;
  }
  return met;
}

// The reads of a stage are in assembly, with their wait: for the compiler they would be reads of LDS that loads into
// the next stage are writing to, and it would wait for those first.

// N fragments of 16 bytes, OFFSET behind the lane's LDS addresses `from`.
template <int OFFSET, int N>
__device__ __forceinline__ void read_keys(const uint32_t* from, half8_t (&k)[N]) {
  static_assert(N == 3 || N == 4, "fragments of a read");
  if constexpr (N == 3)
    asm volatile("ds_read_b128 %0, %3 offset:%6\n\tds_read_b128 %1, %4 offset:%6\n\t"
                 "ds_read_b128 %2, %5 offset:%6\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(k[0]), "=&v"(k[1]), "=&v"(k[2])
                 : "v"(from[0]), "v"(from[1]), "v"(from[2]), "n"(OFFSET)
                 : "memory");
  else
    asm volatile("ds_read_b128 %0, %4 offset:%8\n\tds_read_b128 %1, %5 offset:%8\n\t"
                 "ds_read_b128 %2, %6 offset:%8\n\tds_read_b128 %3, %7 offset:%8\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(k[0]), "=&v"(k[1]), "=&v"(k[2]), "=&v"(k[3])
                 : "v"(from[0]), "v"(from[1]), "v"(from[2]), "v"(from[3]), "n"(OFFSET)
                 : "memory");
}

// Values of 16 keys and 32 N channels as first operands, OFFSET behind the lane's addresses `from` of each 32 channels:
// lane l of 16 reads four channels 4 (l % 4) of key l / 4 and gets channel l of four keys; rows of ROW bytes.
template <int OFFSET, int ROW, int N>
__device__ __forceinline__ void read_values(const uint32_t (&from)[N], half8_t (&v)[N]) {
  static_assert(N >= 2 && N <= 4, "channels of a read");
  typedef short short8_t __attribute__((ext_vector_type(8)));
  short4_t lo[4], hi[4];
  if constexpr (N == 2)
    asm volatile("ds_read_b64_tr_b16 %0, %4 offset:%6\n\tds_read_b64_tr_b16 %1, %4 offset:%7\n\t"
                 "ds_read_b64_tr_b16 %2, %5 offset:%6\n\tds_read_b64_tr_b16 %3, %5 offset:%7\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(lo[1]), "=&v"(hi[1])
                 : "v"(from[0]), "v"(from[1]), "n"(OFFSET), "n"(OFFSET + 8 * ROW)
                 : "memory");
  if constexpr (N == 3)
    asm volatile("ds_read_b64_tr_b16 %0, %6 offset:%9\n\tds_read_b64_tr_b16 %1, %6 offset:%10\n\t"
                 "ds_read_b64_tr_b16 %2, %7 offset:%9\n\tds_read_b64_tr_b16 %3, %7 offset:%10\n\t"
                 "ds_read_b64_tr_b16 %4, %8 offset:%9\n\tds_read_b64_tr_b16 %5, %8 offset:%10\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(lo[1]), "=&v"(hi[1]), "=&v"(lo[2]), "=&v"(hi[2])
                 : "v"(from[0]), "v"(from[1]), "v"(from[2]), "n"(OFFSET), "n"(OFFSET + 8 * ROW)
                 : "memory");
  if constexpr (N == 4)
    asm volatile("ds_read_b64_tr_b16 %0, %8 offset:%12\n\tds_read_b64_tr_b16 %1, %8 offset:%13\n\t"
                 "ds_read_b64_tr_b16 %2, %9 offset:%12\n\tds_read_b64_tr_b16 %3, %9 offset:%13\n\t"
                 "ds_read_b64_tr_b16 %4, %10 offset:%12\n\tds_read_b64_tr_b16 %5, %10 offset:%13\n\t"
                 "ds_read_b64_tr_b16 %6, %11 offset:%12\n\tds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(lo[1]), "=&v"(hi[1]), "=&v"(lo[2]), "=&v"(hi[2]), "=&v"(lo[3]), "=&v"(hi[3])
                 : "v"(from[0]), "v"(from[1]), "v"(from[2]), "v"(from[3]), "n"(OFFSET), "n"(OFFSET + 8 * ROW)
                 : "memory");
#pragma unroll
  for (int b = 0; b < N; ++b)
    v[b] = __builtin_bit_cast(half8_t, short8_t{lo[b][0], lo[b][1], lo[b][2], lo[b][3], hi[b][0], hi[b][1], hi[b][2],
                                                hi[b][3]});
}

// A lane's addresses in LDS: of its fragments of the keys (swizzling moves chunks within 16: the next 16 are 256 bytes
// on) and of the values' 32 channels each, in a stage whose first byte is at `base`; another block or stage is an
// offset in the instruction.
template <int D>
struct Addresses {
  using T = Tile<D>;
  static constexpr int KEYS = D < 128 ? D / 16 : 8, VALUES = D / 32 <= 4 ? D / 32 : 4;
  uint32_t key[KEYS], value[VALUES];
  __device__ __forceinline__ Addresses(uint32_t base, int lane) {
    const int row = lane & 31, half = lane >> 5, swz = T::key_swizzle(row) ^ half;
#pragma unroll
    for (int j = 0; j < KEYS; ++j) key[j] = base + row * T::ROW + 16 * ((2 * j) ^ swz);
    const int l = lane & 15, chunk = 2 * ((lane >> 4) & 1) + ((l & 3) >> 1), vswz = T::value_swizzle(l >> 2);
#pragma unroll
    for (int b = 0; b < VALUES; ++b)
      value[b] = base + (4 * half + (l >> 2)) * T::ROW + 8 * (l & 1) + 16 * ((4 * b + chunk) ^ vswz);
  }
};

// f(I), f(I + STEP), ... below END, with constants.
template <int I, int END, int STEP, typename F>
__device__ __forceinline__ void each(F f) {
  if constexpr (I < END) {
    f(std::integral_constant<int, I>{});
    each<I + STEP, END, STEP>(f);
  }
}

// One block of 32 tokens, whose keys are K and whose values V bytes behind the lane's addresses.  `strange`: rows of
// the values that hold values taken out by hide_strange; value_of(k): where row k of them is in the cache.
template <int D, int K, int V, typename ValueOf>
__device__ __forceinline__ void attend_block(const Addresses<D>& at, const Queries<D>& q, float c, const Seen& seen,
                                             uint32_t strange, ValueOf value_of, Gathered<D>& g) {
  using T = Tile<D>;
  const int lane = __lane_id(), row = lane & 31, half = lane >> 5;
  // scores, a few fragments of the keys at a time: the next are read while the matrix cores have these
  float16_t s = float16_t(0.0f);
  {
    constexpr int N = D == 96 ? 3 : 4;
    auto part = [&](auto j0c) __attribute__((always_inline)) {
      constexpr int j0 = decltype(j0c)::value;
      half8_t k[N];
      if constexpr (Queries<D>::BYTES > 0) {
        half8_t x[N];
        const uint32_t base = (uint32_t)(uintptr_t)q.at;
        const uint32_t queries[4] = {base, base + 1024, base + 2048, base + 3072};
        read_keys<1024 * j0, N>(queries, x);
        read_keys<K + 32 * (j0 / 8 * 8), N>(at.key + j0 % 8, k);
#pragma unroll
        for (int j = 0; j < N; ++j) s = __builtin_amdgcn_mfma_f32_32x32x16_f16(k[j], x[j], s, 0, 0, 0);
        asm volatile("" ::"v"(x[0]));
      } else {
        read_keys<K, N>(at.key + j0, k);
#pragma unroll
        for (int j = 0; j < N; ++j) s = __builtin_amdgcn_mfma_f32_32x32x16_f16(k[j], q.part[j0 + j], s, 0, 0, 0);
      }
      // With a constant zero as its addend, the compiler may give a matrix instruction a destination that overlaps
      // its operands, which this one (8 passes) writes before it has read them all: they stay alive past it.
      asm volatile("" ::"v"(k[0]));
    };
    each<0, D / 16, N>(part);
  }
  // the values' first 16 keys, while the last scores are being made
  constexpr int N = D / 32 <= 4 ? D / 32 : 4, PARTS = D / 32 / N;
  half8_t v[N];
  read_values<V, T::ROW, N>(at.value, v);
  if (!seen.all) {
    const int limit0 = seen.limit0 - 4 * half, limit1 = seen.limit1 - 4 * half;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      s[i] = 8 * ((i >> 2) & 1) + (i & 3) > (i < 8 ? limit0 : limit1) ? -INFINITY : s[i];
  }
  float m = s[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) m = fmaxf(m, s[i]);
  m = both_halves_max(m);
  if (__any((m - g.top) * c > kLag)) {  // (a first score: infinitely above; none yet: NaN, no)
    const float top = fmaxf(m, g.top);
    const float carry = g.top == top ? 1.0f : __builtin_amdgcn_exp2f((g.top - top) * c);
    g.top = top;
    g.sum *= carry;
#pragma unroll
    for (int b = 0; b < D / 32; ++b) g.sums[b] *= carry;
  }
  const float base = g.top == -INFINITY ? 0.0f : g.top * c;
  half8_t p[2];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -base));
    sum += w;
    p[i >> 3][i & 7] = (_Float16)w;
  }
  g.sum += sum;
  each<0, 2 * PARTS, 1>([&](auto ic) __attribute__((always_inline)) {
    constexpr int i = decltype(ic)::value, step = i / PARTS, part = i % PARTS;
    if constexpr (i > 0) read_values<V + 16 * step * T::ROW + 256 * part, T::ROW, N>(at.value, v);
#pragma unroll
    for (int b = 0; b < N; ++b)
      g.sums[part * N + b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v[b], p[step], g.sums[part * N + b], 0, 0, 0);
  });
  while (__builtin_expect(strange != 0, 0)) {
    const int k = __builtin_ctz(strange), in16 = k & 15;
    strange &= strange - 1;
    const int i8 = 4 * ((k >> 3) & 1) + (k & 3);  // of the eight weights of its 16 keys, in lane half (k / 4) % 2
    float w = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) w = i == i8 + 8 * (k >> 4) ? (float)p[i >> 3][i & 7] : w;
    w = __shfl(w, row + 32 * ((k >> 2) & 1));
    const bool sees = in16 <= (k < 16 ? seen.limit0 : seen.limit1);
    const _Float16* from = value_of(k) + 4 * half;
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const half4_t x = *reinterpret_cast<const half4_t*>(from + 32 * b + 8 * n);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool gives = sees && !finite16(__builtin_bit_cast(uint16_t, (_Float16)x[i]));
          g.sums[b][4 * n + i] += gives ? w * (float)x[i] : 0.0f;
        }
        __builtin_amdgcn_sched_barrier(0);
      }
  }
}

}  // namespace awq
