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

// 16 bytes per lane from `base` + the lane's `offset` into LDS, lane after lane.  In assembly, so that the compiler does
// not wait for it before it reads another part of the ring: the waits (vmcnt) stand where the stages change.  (Nothing
// comes back into registers.  The ring's address goes in as well: to the compiler this writes to it.)
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t offset, lds_char* to) {
  uint32_t kept;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3\n\ts_mov_b32 m0, %0"
               : "=&s"(kept)
               : "s"(to), "v"(offset), "s"(base)
               : "memory");
}
// (the count is of loads, in the order of their issue)
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
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

template <int OFFSET>
__device__ __forceinline__ half8_t read16(uint32_t at) {
  return *(const AWQ_LDS half8_t*)(uintptr_t)(at + OFFSET);
}
// Four channels of a row per lane, swapped among 16 lanes: lane l of 16 points to channels 4 (l % 4) of key l / 4 and
// gets channel l of the four keys; and of those 8 rows on.
template <int OFFSET, int ROW>
__device__ __forceinline__ half8_t read_turned(uint32_t at) {
  typedef short short8_t __attribute__((ext_vector_type(8)));
  typedef AWQ_LDS short4_t* lds4;
  const short4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(uintptr_t)(at + OFFSET));
  const short4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(uintptr_t)(at + OFFSET + 8 * ROW));
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

// Fragment j of 32 keys, K bytes behind the lane's addresses, and of the queries.
template <int D, int K, int J>
__device__ __forceinline__ half8_t key_part(const Addresses<D>& at) {
  return read16<K + 32 * (J / 8 * 8)>(at.key[J % 8]);
}
template <int D, int J>
__device__ __forceinline__ half8_t query_part(const Queries<D>& q) {
  if constexpr (Queries<D>::BYTES > 0) return read16<1024 * J>((uint32_t)(uintptr_t)q.at);
  else return q.part[J];
}
// Channels 32 b .. + 31 of 16 of 32 keys, V bytes behind the lane's addresses: I = (D / 32) (16 keys) + b.
template <int D, int V, int I>
__device__ __forceinline__ half8_t value_part(const Addresses<D>& at) {
  constexpr int ROW = Tile<D>::ROW, step = I / (D / 32), b = I % (D / 32);
  return read_turned<V + 16 * step * ROW + 256 * (b / 4), ROW>(at.value[b % 4]);
}

constexpr int kAhead = 4;  // fragments on their way from LDS

// Scores of 32 keys, K bytes behind the lane's addresses: lane (row, half) has keys 8 (i / 4) + 4 half + i % 4.
// beside(j): vector instructions for after matrix instruction j.
template <int D, int K, typename Beside>
__device__ __forceinline__ float16_t scores_of(const Addresses<D>& at, const Queries<D>& q, Beside beside) {
  float16_t s = float16_t(0.0f);
  half8_t k[kAhead], x[kAhead];
  each<0, kAhead, 1>([&](auto jc) __attribute__((always_inline)) {
    constexpr int j = decltype(jc)::value;
    k[j] = key_part<D, K, j>(at);
    x[j] = query_part<D, j>(q);
  });
  in_order();
  each<0, D / 16, 1>([&](auto jc) __attribute__((always_inline)) {
    constexpr int j = decltype(jc)::value, n = j % kAhead;
    s = __builtin_amdgcn_mfma_f32_32x32x16_f16(k[n], x[n], s, 0, 0, 0);
    if constexpr (j == 0) outlive(k[n], x[n]);
    if constexpr (j + kAhead < D / 16) {
      k[n] = key_part<D, K, j + kAhead>(at);
      x[n] = query_part<D, j + kAhead>(q);
    }
    beside(jc);
    in_order();
  });
  return s;
}

// Greatest of 32 scores, of lane and partner.
__device__ __forceinline__ float greatest(const float16_t& s) {
  float m = s[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) m = fmaxf(m, s[i]);
  return both_halves_max(m);
}

// Masks 32 scores, whose greatest is `m` before that, and moves the maximum on; returns what is taken off each, in
// powers of two.
template <int D>
__device__ __forceinline__ float settle(float16_t& s, float m, float c, const Seen& seen, Gathered<D>& g) {
  if (!seen.all) {
    const int half = __lane_id() >> 5, limit0 = seen.limit0 - 4 * half, limit1 = seen.limit1 - 4 * half;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      s[i] = 8 * ((i >> 2) & 1) + (i & 3) > (i < 8 ? limit0 : limit1) ? -INFINITY : s[i];
    m = greatest(s);
  }
  if (__any((m - g.top) * c > kLag)) {  // (a first score: infinitely above; none yet: NaN, no)
    const float top = fmaxf(m, g.top);
    const float carry = g.top == top ? 1.0f : __builtin_amdgcn_exp2f((g.top - top) * c);
    g.top = top;
    g.sum *= carry;
#pragma unroll
    for (int b = 0; b < D / 32; ++b) g.sums[b] *= carry;
  }
  return g.top == -INFINITY ? 0.0f : g.top * c;
}

// The weights of 32 scores as the values' second operand.
struct Weights {
  half8_t part[2];
  float sum = 0.0f;
  // of scores 2 i and 2 i + 1
  __device__ __forceinline__ void take(int i, const float16_t& s, float c, float base) {
    const float w0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * i], c, -base));
    const float w1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * i + 1], c, -base));
    sum += w0 + w1;
    part[i >> 2][2 * (i & 3)] = (_Float16)w0;
    part[i >> 2][2 * (i & 3) + 1] = (_Float16)w1;
  }
};

// The values of 32 keys, V bytes behind the lane's addresses, by their weights.  The first fragments `v` are on their
// way; beside(i): vector instructions for after matrix instruction i.
template <int D, int V>
__device__ __forceinline__ void first_values(const Addresses<D>& at, half8_t (&v)[kAhead]) {
  constexpr int N = 2 * (D / 32) < kAhead ? 2 * (D / 32) : kAhead;
  each<0, N, 1>([&](auto ic) __attribute__((always_inline)) { v[decltype(ic)::value] = value_part<D, V, decltype(ic)::value>(at); });
}
template <int D, int V, typename Beside>
__device__ __forceinline__ void gather(const Addresses<D>& at, half8_t (&v)[kAhead], const Weights& p, Gathered<D>& g,
                                       Beside beside) {
  each<0, 2 * (D / 32), 1>([&](auto ic) __attribute__((always_inline)) {
    constexpr int i = decltype(ic)::value, step = i / (D / 32), b = i % (D / 32);
    g.sums[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v[i % kAhead], p.part[step], g.sums[b], 0, 0, 0);
    if constexpr (i + kAhead < 2 * (D / 32)) v[i % kAhead] = value_part<D, V, i + kAhead>(at);
    beside(ic);
    in_order();
  });
}

// Scores, weights and values of one block after the other: keys K, values V bytes behind the lane's addresses.
template <int D, int K, int V>
__device__ __forceinline__ Weights attend_block(const Addresses<D>& at, const Queries<D>& q, float c, const Seen& seen,
                                                Gathered<D>& g) {
  half8_t v[kAhead];
  float16_t s = scores_of<D, K>(at, q, [&](auto jc) __attribute__((always_inline)) {
    if constexpr (decltype(jc)::value == D / 16 - 1) first_values<D, V>(at, v);
  });
  const float base = settle<D>(s, greatest(s), c, seen, g);
  Weights p;
#pragma unroll
  for (int i = 0; i < 8; ++i) p.take(i, s, c, base);
  g.sum += p.sum;
  gather<D, V>(at, v, p, g, [](auto) __attribute__((always_inline)) {});
  return p;
}

// The same, a block ahead with the scores: the weights of the block whose scores are `s`, with values V bytes behind the
// lane's addresses, beside the products for the next block's scores (keys K bytes behind), and the greatest of
// those, `m`, beside the products with the values.
template <int D, int K, int V>
__device__ __forceinline__ Weights attend_next(const Addresses<D>& at, const Queries<D>& q, float c, const Seen& seen,
                                               float16_t& s, float& m, Gathered<D>& g) {
  constexpr int N = D / 16, M = 2 * (D / 32);
  half8_t v[kAhead];
  Weights p;
  const float base = settle<D>(s, m, c, seen, g);
  in_order();
  float16_t next = scores_of<D, K>(at, q, [&](auto jc) __attribute__((always_inline)) {
    constexpr int j = decltype(jc)::value;
    if constexpr (j == N - 1) first_values<D, V>(at, v);
#pragma unroll
    for (int i = 8 * j / N; i < 8 * (j + 1) / N; ++i) p.take(i, s, c, base);
  });
  g.sum += p.sum;
  float most = -INFINITY;
  gather<D, V>(at, v, p, g, [&](auto ic) __attribute__((always_inline)) {
    constexpr int i = decltype(ic)::value;
#pragma unroll
    for (int n = 8 * i / M; n < 8 * (i + 1) / M; ++n) most = fmaxf(most, fmaxf(next[2 * n], next[2 * n + 1]));
  });
  s = next;
  m = both_halves_max(most);
  return p;
}

// The values that hide_strange took out of rows `strange` of the block, by their weights, to the rows that see them;
// value_of(k): where row k of them is in the cache.
template <int D, typename ValueOf>
__device__ __forceinline__ void gather_strange(uint32_t strange, const Weights& p, const Seen& seen, ValueOf value_of,
                                               Gathered<D>& g) {
  const int lane = __lane_id(), row = lane & 31, half = lane >> 5;
#pragma unroll 1
  while (strange != 0) {
    const int k = __builtin_ctz(strange);
    strange &= strange - 1;
    const int i8 = 4 * ((k >> 3) & 1) + (k & 3);  // of the eight weights of its 16 keys, in lane half (k / 4) % 2
    float w = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) w = i == i8 + 8 * (k >> 4) ? (float)p.part[i >> 3][i & 7] : w;
    w = __shfl(w, row + 32 * ((k >> 2) & 1));
    const bool sees = (k & 15) <= (k < 16 ? seen.limit0 : seen.limit1);
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
