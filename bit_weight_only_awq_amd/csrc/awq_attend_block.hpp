// Shared by the attention kernels: 32 rows of queries (or 16, where there are no
// more) against 32 keys on the matrix cores.
//
// Mathematics: a wave keeps, for each of its 32 rows, the running maximum m of the
// scores, the sum l of the weights 2^((score - m) c) with c = scale log2(e), and
// the weighted sum of the values, one pass over the keys.  Scores are formed
// transposed, keys x queries, so that a lane holds 16 scores of one row (lane %
// 32) and its partner 32 lanes away the other 16 (of 16 rows: 8, and three
// partners): maximum and sum need one exchange (two), and a change of the maximum
// scales a lane's sums by a number it has.  The weights, rounded to fp16, are then in
// place as the second operand of the product with the values, whose first operand
// comes out of LDS transposed; both follow the same order of keys (lane half h holds
// keys 8 j + 4 h .. + 3, lane quarter h of 16 rows keys 16 j + 4 h .. + 3), so nothing is exchanged.  Sums are fp32.
//
// The maximum lags: sums are rescaled only once a score passes it by a factor of
// 2^8, which fp16 holds for weights and fp32 for sums.
//
// The weights' rounding is to what the matrix cores multiply (bf16 would be 2^-9).  They are held 2^7 times as large (up
// to 2^15 with the lag, of fp16's 2^16): relative 2^-11 down to 2^-21 of the maximum, below that 2^-32 of it at most, so
// that 2^17 keys of 2^-26 of a great one still count.  l is the sum of the rounded weights: the result is an average of
// the values, and no channel passes the greatest of them.  (With l of the weights before rounding, 2000 values of 65504 gave
// infinity; products of two halves by 1 and 1 add eight of them up now: 13 questions 520 -> 527 us, prompt of 2000: 50.7 ->
// 51.0, single tokens the same.)
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
constexpr float kLag = 8.0f;   // the maximum lags by at most this power of two
constexpr float kLift = 7.0f;  // the weights are held this power of two larger
constexpr float kFar = 1024.0f;  // past this power of two what is taken off is not rounded into one number

// Rows of D halves in LDS, as 16-byte chunks: chunk c of row r is at chunk c ^ swizzle(r), so that what
// half a wave reads in one instruction lies in different banks (16 rows of one chunk for keys; for values 4 rows of 4
// chunks, or 8 rows of 2).
template <int D>
struct Tile {
  static constexpr int CHUNKS = D / 8, ROW = D * 2;
  static constexpr int LOADS = D / 32;  // loads of 64 chunks per 16 rows
  static __device__ __forceinline__ int key_swizzle(int r) {
    return D == 64 ? (r >> 1) & 7 : D == 96 ? (r >> 2) & 3 : r & 15;
  }
  static __device__ __forceinline__ int value_swizzle(int r) {
    const int fours = ((r >> 2) & 1) << 1;
    return D == 64 ? ((r >> 1) & 1) << 2 | fours : D == 96 ? fours : (r & 3) << 2 | fours;
  }
};

// Where a lane reads from, in bytes from the first of 16 rows, for each of the loads of 64 chunks that bring them:
// the chunks' swizzles are powers of two apart from load to load (but not of rows of 12 chunks).
template <int D>
struct Sources {
  using T = Tile<D>;
  static constexpr int KEPT = D == 96 ? 3 : 1, ROWS = 64 / T::CHUNKS;
  uint32_t keys[KEPT], values[KEPT];
  __device__ __forceinline__ explicit Sources(int lane) {
#pragma unroll
    for (int i = 0; i < KEPT; ++i) {
      const int at = 64 * i + lane, r = at / T::CHUNKS, c = at % T::CHUNKS;
      keys[i] = (uint32_t)(r * T::ROW + 16 * (c ^ T::key_swizzle(r)));
      values[i] = (uint32_t)(r * T::ROW + 16 * (c ^ T::value_swizzle(r)));
    }
  }
  __device__ __forceinline__ uint32_t key(int i) const {
    return D == 96 ? keys[i] : (keys[0] ^ (uint32_t)(16 * (D == 64 ? 4 * i : ROWS * i))) + 1024 * i;
  }
  __device__ __forceinline__ uint32_t value(int i) const {
    return D == 96 ? values[i]
                   : (values[0] ^ (uint32_t)(D == 256 ? 128 * (i & 1) + 16 * (i & 2) : D == 128 ? 32 * (i & 1) : 0)) + 1024 * i;
  }
};

// N times 64 times 16 bytes, from `base` + the lane's `offset`s, into LDS from `to` on, lane after lane.  In assembly, so
// that the compiler does not wait for it before it reads another part of the ring: the waits (vmcnt) stand where the
// blocks change.  (Nothing comes back into registers.  The ring's address goes in as well: to the compiler this writes
// to it.)
template <int N>
__device__ __forceinline__ void load_to_lds(const char* base, const uint32_t (&offset)[N], lds_char* to) {
  static_assert(N >= 1 && N <= 4, "loads of 16 rows, or some of them");
  uint32_t kept;
  if constexpr (N == 1)
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %3, %2\n\ts_mov_b32 m0, %0"
                 : "=&s"(kept)
                 : "s"(to), "s"(base), "v"(offset[0])
                 : "memory");
  if constexpr (N == 2)
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %3, %2\n\t"
                 "s_add_u32 m0, m0, 1024\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %4, %2\n\ts_mov_b32 m0, %0"
                 : "=&s"(kept)
                 : "s"(to), "s"(base), "v"(offset[0]), "v"(offset[1])
                 : "memory", "scc");
  if constexpr (N == 3)
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %3, %2\n\t"
                 "s_add_u32 m0, m0, 1024\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %4, %2\n\t"
                 "s_add_u32 m0, m0, 1024\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %5, %2\n\ts_mov_b32 m0, %0"
                 : "=&s"(kept)
                 : "s"(to), "s"(base), "v"(offset[0]), "v"(offset[1]), "v"(offset[2])
                 : "memory", "scc");
  if constexpr (N == 4)
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %3, %2\n\t"
                 "s_add_u32 m0, m0, 1024\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %4, %2\n\t"
                 "s_add_u32 m0, m0, 1024\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %5, %2\n\t"
                 "s_add_u32 m0, m0, 1024\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %6, %2\n\ts_mov_b32 m0, %0"
                 : "=&s"(kept)
                 : "s"(to), "s"(base), "v"(offset[0]), "v"(offset[1]), "v"(offset[2]), "v"(offset[3])
                 : "memory", "scc");
}
// (the count is of loads, in the order of their issue)
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The larger of two, NaN if either is: one instruction for three numbers, where the maximum that passes NaN over takes
// one more for each.  (A row with a NaN among its scores is NaN, whatever its maximum.)
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Greatest and sum over the lanes that share a row (R rows: lane % R).
template <int R>
__device__ __forceinline__ float row_max(float v) {
  if constexpr (R == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false,
                                                    false);
    const uint32_t r0 = r[0], r1 = r[1];
    v = larger(__builtin_bit_cast(float, r0), __builtin_bit_cast(float, r1));
  }
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false,
                                                  false);
  const uint32_t r0 = r[0], r1 = r[1];
  return larger(__builtin_bit_cast(float, r0), __builtin_bit_cast(float, r1));
}
template <int R>
__device__ __forceinline__ float row_sum(float v) {
  if constexpr (R == 16) v = swap_sum16(v, v);
  return swap_sum32(v, v);
}

// Scores of 32 keys and R rows, and what R rows gather: in a lane of row lane % R and part h = lane / R, scores 4 i .. 4
// i + 3 are of keys (256 / R) i + 4 h .. + 3, sums 4 n .. 4 n + 3 of channels (256 / R) n + 4 h .. + 3.
template <int R>
struct Scores;
template <>
struct Scores<32> {
  static constexpr int COUNT = 16;
  float16_t s;
  __device__ __forceinline__ float get(int i) const { return s[i]; }
  __device__ __forceinline__ void put(int i, float v) { s[i] = v; }
};
template <>
struct Scores<16> {
  static constexpr int COUNT = 8;
  float4_t s[2];
  __device__ __forceinline__ float get(int i) const { return s[i >> 2][i & 3]; }
  __device__ __forceinline__ void put(int i, float v) { s[i >> 2][i & 3] = v; }
};

// Where a head is 256 wide, the sums stay in the accumulator half of the registers, which only matrix instructions work
// in: left to itself the compiler moves all of them to the other half and back for every block, because now and then
// they are scaled.  `apart` stands between matrix instructions and those that touch single sums: it waits for the
// former's results (at most 19 cycles after one of 16 passes) and for the latter's.
template <int N, typename V>
__device__ __forceinline__ void apart(V (&sums)[N]) {
  if constexpr (N == 8)
    asm volatile("s_nop 15\n\ts_nop 7"
                 : "+a"(sums[0]), "+a"(sums[1]), "+a"(sums[2]), "+a"(sums[3]), "+a"(sums[4]), "+a"(sums[5]), "+a"(sums[6]),
                   "+a"(sums[7]));
  else {
    static_assert(N == 16, "256 channels");
    asm volatile("s_nop 15\n\ts_nop 7"
                 : "+a"(sums[0]), "+a"(sums[1]), "+a"(sums[2]), "+a"(sums[3]), "+a"(sums[4]), "+a"(sums[5]), "+a"(sums[6]),
                   "+a"(sums[7]), "+a"(sums[8]), "+a"(sums[9]), "+a"(sums[10]), "+a"(sums[11]), "+a"(sums[12]),
                   "+a"(sums[13]), "+a"(sums[14]), "+a"(sums[15]));
  }
}
__device__ __forceinline__ float scaled_apart(float sum, float by) {
  float t;
  asm("v_accvgpr_read_b32 %1, %0\n\tv_mul_f32 %1, %1, %2\n\tv_accvgpr_write_b32 %0, %1" : "+a"(sum), "=&v"(t) : "v"(by));
  return sum;
}
__device__ __forceinline__ float added_apart(float sum, float x) {
  float t;
  asm("v_accvgpr_read_b32 %1, %0\n\tv_add_f32 %1, %1, %2\n\tv_accvgpr_write_b32 %0, %1" : "+a"(sum), "=&v"(t) : "v"(x));
  return sum;
}

template <int D, int R>
struct Gathered;
template <int D>
struct Gathered<D, 32> {
  static constexpr int QUADS = D / 8;
  float16_t sums[D / 32];
  float top, sum;  // the maximum; the lane's share of l
  __device__ __forceinline__ float get(int n, int i) const { return sums[n >> 2][4 * (n & 3) + i]; }
  __device__ __forceinline__ void pause() {
    if constexpr (D == 256) apart(sums);
  }
  __device__ __forceinline__ void add(int n, int i, float v) {
    const float sum = get(n, i);
    sums[n >> 2][4 * (n & 3) + i] = D == 256 ? added_apart(sum, v) : sum + v;
  }
  __device__ __forceinline__ void scale(float by) {
    pause();
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
      if constexpr (D < 256) {
        sums[b] *= by;
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) sums[b][i] = scaled_apart(sums[b][i], by);
      }
    }
    pause();
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int b = 0; b < D / 32; ++b) sums[b] = float16_t(0.0f);
    top = -INFINITY;
    sum = 0.0f;
  }
};
template <int D>
struct Gathered<D, 16> {
  static constexpr int QUADS = D / 16;
  float4_t sums[QUADS];
  float top, sum;
  __device__ __forceinline__ float get(int n, int i) const { return sums[n][i]; }
  __device__ __forceinline__ void pause() {
    if constexpr (D == 256) apart(sums);
  }
  __device__ __forceinline__ void add(int n, int i, float v) {
    sums[n][i] = D == 256 ? added_apart(sums[n][i], v) : sums[n][i] + v;
  }
  __device__ __forceinline__ void scale(float by) {
    pause();
#pragma unroll
    for (int n = 0; n < QUADS; ++n) {
      if constexpr (D < 256) {
        sums[n] *= by;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[n][i] = scaled_apart(sums[n][i], by);
      }
    }
    pause();
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < QUADS; ++n) sums[n] = float4_t(0.0f);
    top = -INFINITY;
    sum = 0.0f;
  }
};

// Fragments of R rows' queries: row lane % R, channels 8 (64 / R) j + 8 (lane / R) .. + 7.
template <int D, int R>
struct Queries {
  static constexpr int PARTS = D * R / 512;
  half8_t part[PARTS];
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

// A lane's addresses in LDS: of its fragments of the keys and of the values' channels (swizzling moves chunks within
// 16: the next 16 are 256 bytes on), in a block whose first byte is at `base`; another block is an offset in the
// instruction.
template <int D, int R>
struct Addresses {
  using T = Tile<D>;
  static constexpr int WIDE = D < 128 ? D : 128, KEYS = WIDE * R / 512, VALUES = WIDE / R;
  uint32_t key[KEYS], value[VALUES];
  __device__ __forceinline__ Addresses(uint32_t base, int lane) {
    const int row = lane & (R - 1), h = lane / R, swz = T::key_swizzle(row) ^ h;
#pragma unroll
    for (int j = 0; j < KEYS; ++j) key[j] = base + row * T::ROW + 16 * ((64 / R * j) ^ swz);
    // 16 lanes point to 4 rows of 16 channels: of 32 rows' values, the next 16 lanes to the next 16 channels
    const int l = lane & 15, from = 4 * h + (l >> 2), chunk = (R == 32 ? 2 * ((lane >> 4) & 1) : 0) + ((l & 3) >> 1);
#pragma unroll
    for (int b = 0; b < VALUES; ++b)
      value[b] = base + from * T::ROW + 8 * (l & 1) + 16 * ((R / 8 * b + chunk) ^ T::value_swizzle(from));
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

template <int OFFSET>
__device__ __forceinline__ half8_t read16(uint32_t at) {
  return *(const AWQ_LDS half8_t*)(uintptr_t)(at + OFFSET);
}
// Four channels of a row per lane, swapped among 16 lanes: lane l of 16 points to channels 4 (l % 4) of key l / 4 and
// gets channel l of the four keys; and of those APART bytes on.
template <int OFFSET, int APART>
__device__ __forceinline__ half8_t read_turned(uint32_t at) {
  typedef short short8_t __attribute__((ext_vector_type(8)));
  typedef AWQ_LDS short4_t* lds4;
  const short4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(uintptr_t)(at + OFFSET));
  const short4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(uintptr_t)(at + OFFSET + APART));
  return __builtin_bit_cast(half8_t, short8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
}

// The order of the instructions below is the order of the source, step by step: left to itself the compiler reads a
// fragment, waits for it and multiplies, one after the other, and keeps vector instructions apart from matrix ones.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// With a constant zero as its addend, the compiler may give a matrix instruction a destination that overlaps its
// operands, which this one (8 passes) writes before it has read them all: they stay alive past it.
__device__ __forceinline__ void outlive(half8_t a, half8_t b) {
  in_order();
  asm volatile("" ::"v"(a), "v"(b));
}

// The products of a block, in order.  Scores: fragment J of the keys with fragment J % PARTS of the queries (of 16 rows,
// the first 16 keys, then the others).  Values: I = (D / 32) (16 keys) + 32 channels; of 16 rows: 16 channels, all keys.
template <int D, int R>
struct Products {
  static constexpr int SCORES = D / 16, VALUES = D / 16, PARTS = Queries<D, R>::PARTS;
};
template <int D, int R, int K, int J>
__device__ __forceinline__ half8_t key_part(const Addresses<D, R>& at) {
  constexpr int PARTS = Queries<D, R>::PARTS, KEYS = Addresses<D, R>::KEYS, j = J % PARTS;
  return read16<K + J / PARTS * 16 * Tile<D>::ROW + 256 * (j / KEYS)>(at.key[j % KEYS]);
}
template <int D, int R, int V, int I>
__device__ __forceinline__ half8_t value_part(const Addresses<D, R>& at) {
  constexpr int ROW = Tile<D>::ROW, VALUES = Addresses<D, R>::VALUES;
  constexpr int b = R == 32 ? I % (D / 32) : I, rows = R == 32 ? 16 * (I / (D / 32)) : 0;
  return read_turned<V + rows * ROW + 256 * (b / VALUES), (R == 32 ? 8 : 16) * ROW>(at.value[b % VALUES]);
}

constexpr int kAhead = 4;  // fragments on their way from LDS

struct Fragments {
  half8_t k[kAhead];
};
template <int D, int R, int K>
__device__ __forceinline__ Fragments first_keys(const Addresses<D, R>& at) {
  Fragments f;
  each<0, kAhead, 1>([&](auto jc) __attribute__((always_inline)) {
    constexpr int j = decltype(jc)::value;
    f.k[j] = key_part<D, R, K, j>(at);
  });
  return f;
}

// Scores of 32 keys, K bytes behind the lane's addresses, the first fragments on their way.  beside(j): vector
// instructions for after matrix instruction j.
template <int D, int R, int K, typename Beside>
__device__ __forceinline__ Scores<R> scores_of(const Addresses<D, R>& at, const Queries<D, R>& q, Fragments& f,
                                               Beside beside) {
  using P = Products<D, R>;
  Scores<R> s{};
  auto& k = f.k;
  in_order();
  each<0, P::SCORES, 1>([&](auto jc) __attribute__((always_inline)) {
    constexpr int j = decltype(jc)::value, n = j % kAhead;
    const half8_t x = q.part[j % P::PARTS];
    if constexpr (R == 32) s.s = __builtin_amdgcn_mfma_f32_32x32x16_f16(k[n], x, s.s, 0, 0, 0);
    else s.s[j / P::PARTS] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[n], x, s.s[j / P::PARTS], 0, 0, 0);
    if constexpr (j % P::PARTS == 0) outlive(k[n], x);
    if constexpr (j + kAhead < P::SCORES) k[n] = key_part<D, R, K, j + kAhead>(at);
    beside(jc);
    in_order();
  });
  return s;
}

// Greatest of a row's 32 scores.
template <int R>
__device__ __forceinline__ float greatest(const Scores<R>& s) {
  float m = s.get(0);
#pragma unroll
  for (int i = 1; i < Scores<R>::COUNT; ++i) m = larger(m, s.get(i));
  return row_max<R>(m);
}

// Masks 32 scores; returns their greatest.
template <int R>
__device__ __forceinline__ float mask(Scores<R>& s, const Seen& seen) {
  const int h = __lane_id() / R, limit0 = seen.limit0 - 4 * h, limit1 = seen.limit1 - 4 * h;
#pragma unroll
  for (int i = 0; i < Scores<R>::COUNT; ++i) {
    const int k = 256 / R * (i >> 2) + (i & 3);
    s.put(i, (k & 15) > (k < 16 ? limit0 : limit1) ? -INFINITY : s.get(i));
  }
  return greatest(s);
}

// Moves the maximum on to that of 32 scores, whose greatest is `m`; returns what is taken off each, in powers of two.  (Every
// part of a row is lifted alike, so that nothing has to be taken off again where parts are joined.)  That number is rounded,
// which up to kFar is nothing beside a weight's own rounding (2^-15 of a power of two: 2e-5); past it the maximum is taken
// off the scores themselves, whose differences are exact: of scores of 10^9 it would be off by more powers of two than a
// weight has.  (The question costs 13 questions 523 -> 526 us, a prompt of 2000 51.2 -> 51.8.)
template <int D, int R>
__device__ __forceinline__ float settle(float m, float c, Scores<R>& s, Gathered<D, R>& g) {
  if (__any((m - g.top) * c > kLag)) {  // (a first score: infinitely above; none yet: NaN, no)
    const float top = m > g.top ? m : g.top;
    const float carry = g.top == top ? 1.0f : __builtin_amdgcn_exp2f((g.top - top) * c);
    g.top = top;
    g.sum *= carry;
    g.scale(carry);
  }
  const float base = __builtin_fmaf(g.top, c, -kLift);
  const bool far = __builtin_fabsf(base) > kFar;
  if (__builtin_expect(!__any(far), 1)) return base;
  const float off = far && g.top != -INFINITY ? g.top : 0.0f;
#pragma unroll
  for (int i = 0; i < Scores<R>::COUNT; ++i) s.put(i, s.get(i) - off);
  return g.top == -INFINITY ? 0.0f : far ? -kLift : base;
}

// The weights of 32 scores as the values' second operand.
template <int R>
struct Weights {
  half8_t part[R / 16];
  float eights[R / 16];  // sums of eight, as rounded (added to l one after the other, they move the scores' registers: two
                         // sets of the three that a loop of row tiles takes in turn then share a pair)
  // of scores 2 i and 2 i + 1
  __device__ __forceinline__ void take(int i, const Scores<R>& s, float c, float base) {
    const half2_t two{(_Float16)__builtin_amdgcn_exp2f(__builtin_fmaf(s.get(2 * i), c, -base)),
                      (_Float16)__builtin_amdgcn_exp2f(__builtin_fmaf(s.get(2 * i + 1), c, -base))};
    eights[i / 4] = __builtin_amdgcn_fdot2(two, half2_t((_Float16)1.0f), i % 4 ? eights[i / 4] : 0.0f, false);
    part[i >> 2][2 * (i & 3)] = two[0];
    part[i >> 2][2 * (i & 3) + 1] = two[1];
  }
};

// The values of 32 keys, V bytes behind the lane's addresses, by their weights.  The first fragments `v` are on their
// way; beside(i): vector instructions for after matrix instruction i.
template <int D, int R, int V>
__device__ __forceinline__ void first_values(const Addresses<D, R>& at, half8_t (&v)[kAhead]) {
  each<0, kAhead, 1>([&](auto ic) __attribute__((always_inline)) {
    v[decltype(ic)::value] = value_part<D, R, V, decltype(ic)::value>(at);
  });
}
template <int D, int R, int V, typename Beside>
__device__ __forceinline__ void gather(const Addresses<D, R>& at, half8_t (&v)[kAhead], const Weights<R>& p,
                                       Gathered<D, R>& g, Beside beside) {
  each<0, Products<D, R>::VALUES, 1>([&](auto ic) __attribute__((always_inline)) {
    constexpr int i = decltype(ic)::value, b = R == 32 ? i % (D / 32) : i, step = R == 32 ? i / (D / 32) : 0;
    if constexpr (R == 32) g.sums[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v[i % kAhead], p.part[step], g.sums[b], 0, 0, 0);
    else g.sums[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[i % kAhead], p.part[step], g.sums[b], 0, 0, 0);
    if constexpr (i + kAhead < Products<D, R>::VALUES) v[i % kAhead] = value_part<D, R, V, i + kAhead>(at);
    beside(ic);
    in_order();
  });
}

// Scores, weights and values of one block after the other: keys K, values V bytes behind the lane's addresses.
template <int D, int R, int K, int V>
__device__ __forceinline__ Weights<R> attend_block(const Addresses<D, R>& at, const Queries<D, R>& q, float c,
                                                   const Seen& seen, Gathered<D, R>& g) {
  half8_t v[kAhead];
  Fragments f = first_keys<D, R, K>(at);
  Scores<R> s = scores_of<D, R, K>(at, q, f, [&](auto jc) __attribute__((always_inline)) {
    if constexpr (decltype(jc)::value == Products<D, R>::SCORES - 1) first_values<D, R, V>(at, v);
  });
  const float base = settle<D, R>(seen.all ? greatest(s) : mask(s, seen), c, s, g);
  Weights<R> p;
#pragma unroll
  for (int i = 0; i < Scores<R>::COUNT / 2; ++i) p.take(i, s, c, base);
#pragma unroll
  for (int i = 0; i < Scores<R>::COUNT / 8; ++i) g.sum += p.eights[i];
  gather<D, R, V>(at, v, p, g, [](auto) __attribute__((always_inline)) {});
  return p;
}

// The same, a block ahead with the scores: the weights of the block whose scores are `s`, with values V bytes behind the
// lane's addresses, beside the products for the next block's scores (keys K bytes behind, the first fragments on their
// way), and the greatest of those, `m`, beside the products with the values, as well as beside(i), after every other of
// them.
template <int D, int R, int K, int V, typename Beside>
__device__ __forceinline__ Weights<R> attend_next(const Addresses<D, R>& at, const Queries<D, R>& q, Fragments& f, float c,
                                                  const Seen& seen, Scores<R>& s, float& m, Gathered<D, R>& g, Beside beside) {
  constexpr int N = Products<D, R>::SCORES, M = Products<D, R>::VALUES, PAIRS = Scores<R>::COUNT / 2;
  half8_t v[kAhead];
  Weights<R> p;
  if (!seen.all) m = mask(s, seen);
  const float base = settle<D, R>(m, c, s, g);
  in_order();
  Scores<R> next = scores_of<D, R, K>(at, q, f, [&](auto jc) __attribute__((always_inline)) {
    constexpr int j = decltype(jc)::value;
    if constexpr (j == N - 2) first_values<D, R, V>(at, v);
#pragma unroll
    for (int i = PAIRS * j / N; i < PAIRS * (j + 1) / N; ++i) p.take(i, s, c, base);
  });
  float most = -INFINITY;
  gather<D, R, V>(at, v, p, g, [&](auto ic) __attribute__((always_inline)) {
    constexpr int i = decltype(ic)::value;
#pragma unroll
    for (int n = PAIRS * i / M; n < PAIRS * (i + 1) / M; ++n) {
      most = larger(larger(most, next.get(2 * n)), next.get(2 * n + 1));
      if (n % 4 == 3) g.sum += p.eights[n / 4];
    }
    if constexpr (i % 2 == 0) beside(std::integral_constant<int, i / 2>{});
  });
  asm volatile("" : "+v"(g.sum));  // (here, beside the matrix instructions, and not after them)
  s = next;
  m = row_max<R>(most);
  return p;
}

// The values that hide_strange took out of rows `strange` of the block, by their weights, to the rows that see them;
// value_of(k): where row k of them is in the cache.
template <int D, int R, typename ValueOf>
__device__ __forceinline__ void gather_strange(uint32_t strange, const Weights<R>& p, const Seen& seen, ValueOf value_of,
                                               Gathered<D, R>& g) {
  const int lane = __lane_id(), row = lane & (R - 1), h = lane / R;
  g.pause();
#pragma unroll 1
  while (strange != 0) {
    const int k = __builtin_ctz(strange);
    strange &= strange - 1;
    // its weight is number `at` of those in part `of` of the lanes
    const int of = (k >> 2) & (64 / R - 1), at = R == 32 ? 4 * (k >> 3) + (k & 3) : 4 * (k >> 4) + (k & 3);
    float w = 0.0f;
#pragma unroll
    for (int i = 0; i < Scores<R>::COUNT; ++i) w = i == at ? (float)p.part[i >> 3][i & 7] : w;
    w = __shfl(w, row + R * of);
    const bool sees = (k & 15) <= (k < 16 ? seen.limit0 : seen.limit1);
    const _Float16* from = value_of(k) + 4 * h;
#pragma unroll
    for (int n = 0; n < Gathered<D, R>::QUADS; ++n) {
      const half4_t x = *reinterpret_cast<const half4_t*>(from + 256 / R * n);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool gives = sees && !finite16(__builtin_bit_cast(uint16_t, (_Float16)x[i]));
        g.add(n, i, gives ? w * (float)x[i] : 0.0f);
      }
      in_order();
    }
  }
  g.pause();
}

}  // namespace awq
