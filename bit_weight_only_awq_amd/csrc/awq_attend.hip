// Attention over a paged cache (awq_attend, awq_attend_pages).
#include "awq_cache.hpp"

namespace awq {
namespace {

// One wave per row and query head: 64 keys at a time, each lane one key's
// product, then each lane its channels of the values.
__global__ __launch_bounds__(64) void attend_simple_kernel(AttendArgs a, CacheArgs c, SeqArgs s) {
  __shared__ float share[64];
  const int lane = threadIdx.x, t = blockIdx.x / a.q_heads, head = blockIdx.x % a.q_heads, D = c.dim, kv = head / (a.q_heads / c.heads);
  const Sequence seq = sequence_of(s, c.shift, t);
  if (seq.rows == 0) return;
  const int place = t - seq.row0 + seq.place0(), S = 1 << c.shift;
  const _Float16* q = a.q + t * a.ldq + (int64_t)head * D;
  const int* table = s.tables + (int64_t)seq.index * s.width;
  const int* list = a.list ? a.list + ((int64_t)t * c.heads + kv) * a.count : nullptr;
  const int64_t keys = list ? (int64_t)a.count << c.shift : (int64_t)place + 1;
  float top = -INFINITY, total = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t j0 = 0; j0 < keys; j0 += 64) {
    const int64_t j = j0 + lane;
    const int entry = (int)(min(j, keys - 1) >> c.shift), slot = (int)(j & (S - 1));
    const int page = list ? list[entry] : entry;
    const bool seen = j < keys && page >= 0 && page < s.width && ((int64_t)page << c.shift) + slot <= place;
    const int64_t at =
        ((((int64_t)(seen ? page_number(c, table[page]) : 0) * c.heads + kv) << c.shift) + slot) * D;
    float score = -INFINITY;
    if (seen) {
      score = 0.0f;
      for (int d = 0; d < D; d += 8) {
        const half8_t x = *reinterpret_cast<const half8_t*>(q + d), y = *reinterpret_cast<const half8_t*>(c.k + at + d);
#pragma unroll
        for (int i = 0; i < 8; ++i) score += (float)x[i] * (float)y[i];
      }
      score *= a.scale * 1.4426950408889634f;
    }
    float m = score;
    for (int x = 1; x < 64; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
    m = fmaxf(m, top);
    const float base = m == -INFINITY ? 0.0f : m, carry = exp2f(top - base);
    const float p = seen ? exp2f(score - base) : 0.0f;
    float sum = p;
    for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x);
    total = total * carry + sum;
    top = m;
    for (int i = 0; i < 4; ++i) acc[i] *= carry;
    const unsigned long long any = __ballot(seen);
    share[lane] = p;
    __syncthreads();
    for (int k = 0; k < 64; ++k) {
      if (!(any >> k & 1)) continue;
      const int64_t row = (int64_t)__shfl((int)(at >> 32), k) << 32 | (uint32_t)__shfl((int)(uint32_t)at, k);
      for (int i = 0; i < 4; ++i)
        if (lane + 64 * i < D) acc[i] += share[k] * (float)c.v[row + lane + 64 * i];
    }
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    if (lane + 64 * i < D)
      a.y[t * a.ldy + (int64_t)head * D + lane + 64 * i] = (_Float16)(total == 0.0f ? 0.0f : acc[i] / total);
}

}  // namespace

size_t attend_workspace_bytes(int, int, int, int, int, int, int, int) { return 0; }
size_t attend_list_workspace_bytes(int, int, int, int, int, int) { return 0; }

hipError_t launch_attend(const AttendArgs& a, const CacheArgs& c, const SeqArgs& s, void*, hipStream_t stream) {
  hipLaunchKernelGGL(attend_simple_kernel, dim3(s.T * a.q_heads), dim3(64), 0, stream, a, c, s);
  return hipGetLastError();
}

}  // namespace awq
