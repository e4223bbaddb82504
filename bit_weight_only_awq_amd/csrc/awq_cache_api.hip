// C ABI of the operators on a paged cache of keys and values: argument
// validation, then the launches on the caller's stream.  The contract of every
// entry point is in include/awq.h.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/awq.h"
#include "awq_launch_cache.hpp"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }  // numbers read one by one

constexpr int32_t kMaxDim = 1 << 21;   // row strides
constexpr int32_t kMaxSeqs = 1 << 16;
constexpr int32_t kMaxHeads = 1024;
constexpr int32_t kMaxRows = 1 << 24;  // tokens times query heads, below it: launches of less than 2^32 threads
constexpr int32_t kMaxChosen = 1 << 22;  // tokens times key heads of a selection, likewise
constexpr int32_t kMaxAxes = 16;

bool dim_known(int32_t dim) { return dim == 64 || dim == 96 || dim == 128 || dim == 256; }
bool page_known(int32_t size) { return size >= 16 && size <= 256 && (size & (size - 1)) == 0; }

// Token and head counts and the tables' width; then the page size, so that places stay within 30 bits.
bool counts_ok(int32_t T, int32_t B, int32_t q_heads, int32_t kv_heads, int32_t width, int32_t page_size) {
  return T >= 1 && B >= 1 && B <= kMaxSeqs && kv_heads >= 1 && q_heads >= kv_heads && q_heads <= kMaxHeads &&
         q_heads % kv_heads == 0 && (int64_t)T * q_heads < kMaxRows && width >= 1 && page_known(page_size) &&
         (int64_t)width * page_size <= ((int64_t)1 << 30);
}

int check_cache(const int32_t* offsets, const int32_t* lengths, const int32_t* tables, int32_t width, int32_t T, int32_t B,
                int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t pages, int32_t page_size) {
  if (!counts_ok(T, B, q_heads, kv_heads, width, page_size) || pages < 1) return AWQ_ERR_SHAPE;
  if (!dim_known(head_dim)) return AWQ_ERR_UNSUPPORTED;
  if (!offsets || !lengths || !tables) return AWQ_ERR_NULL;
  return aligned4(offsets) && aligned4(lengths) && aligned4(tables) ? AWQ_OK : AWQ_ERR_ALIGN;
}

// (the kernels work in powers of two: the scale times log2(e) must be finite as well)
bool scale_ok(float scale) { return scale > 0.0f && !isinf(scale * 1.4426950408889634f); }

bool stride_ok(int32_t ld, int64_t row) { return ld >= row && ld <= kMaxDim && (ld & 7) == 0; }

int check_pointers(const void* a, const void* b, const void* c, const void* d) {
  if (!a || !b || !c || !d) return AWQ_ERR_NULL;
  return aligned16(a) && aligned16(b) && aligned16(c) && aligned16(d) ? AWQ_OK : AWQ_ERR_ALIGN;
}

int check_workspace(const void* workspace, size_t have, size_t need) {
  if (have < need) return AWQ_ERR_WORKSPACE;
  if (need > 0 && !workspace) return AWQ_ERR_NULL;
  return need > 0 && !aligned16(workspace) ? AWQ_ERR_ALIGN : AWQ_OK;
}

int from_hip(hipError_t e) { return e == hipSuccess ? AWQ_OK : AWQ_ERR_HIP; }

// (the kernels read through the same structure that appending writes through)
awq::CacheArgs cache(const void* k, const void* v, const void* bounds, int32_t pages, int32_t heads, int32_t dim,
                     int32_t page_size) {
  auto halves = [](const void* p) { return static_cast<_Float16*>(const_cast<void*>(p)); };
  return awq::CacheArgs{halves(k), halves(v), halves(bounds), pages, heads, dim, __builtin_ctz(page_size)};
}

}  // namespace

extern "C" {

int awq_append_kv(const void* x, int32_t ldx, const int32_t* offsets, const int32_t* lengths, const int32_t* tables,
                  int32_t width, int32_t T, int32_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                  const float* inv_freq, int32_t rotary, int32_t interleaved, const int32_t* positions, int32_t axes,
                  const int32_t* axis, void* q, int32_t ldq, void* k_pages, void* v_pages, void* bounds, int32_t pages,
                  int32_t page_size, void* stream) {
  int st = check_cache(offsets, lengths, tables, width, T, B, q_heads, kv_heads, head_dim, pages, page_size);
  if (st != AWQ_OK) return st;
  if (!stride_ok(ldx, (int64_t)(q_heads + 2 * kv_heads) * head_dim) || !stride_ok(ldq, (int64_t)q_heads * head_dim))
    return AWQ_ERR_SHAPE;
  if (rotary < 0 || rotary > head_dim || rotary % 16 != 0) return AWQ_ERR_OPTION;
  if (positions && (axes < 1 || axes > kMaxAxes)) return AWQ_ERR_OPTION;
  st = check_pointers(x, q, k_pages, v_pages);
  if (st != AWQ_OK) return st;
  if (rotary > 0 && (!inv_freq || (positions && axes > 1 && !axis))) return AWQ_ERR_NULL;
  if (!aligned16(bounds) || !aligned4(inv_freq) || !aligned4(positions) || !aligned4(axis)) return AWQ_ERR_ALIGN;
  const awq::AppendArgs a{static_cast<const _Float16*>(x), ldx, q_heads, inv_freq, rotary, interleaved != 0, positions,
                          axes, axis, static_cast<_Float16*>(q), ldq};
  return from_hip(awq::launch_append(a, cache(k_pages, v_pages, bounds, pages, kv_heads, head_dim, page_size),
                                     awq::SeqArgs{offsets, lengths, tables, width, T, B},
                                     static_cast<hipStream_t>(stream)));
}

size_t awq_attend_workspace_bytes(int32_t T, int32_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                  int32_t width, int32_t page_size, int32_t shared) {
  if (!counts_ok(T, B, q_heads, kv_heads, width, page_size) || !dim_known(head_dim) || shared < 0 ||
      !awq::attend_fits(T, B, q_heads, kv_heads, head_dim, page_size, width, shared))
    return 0;
  return awq::attend_workspace_bytes(T, B, q_heads, kv_heads, head_dim, page_size, width, shared);
}

int awq_attend(const void* q, int32_t ldq, const int32_t* offsets, const int32_t* lengths, const int32_t* tables,
               int32_t width, int32_t T, int32_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim, float scale,
               int32_t shared, const void* k_pages, const void* v_pages, int32_t pages, int32_t page_size, void* y,
               int32_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_cache(offsets, lengths, tables, width, T, B, q_heads, kv_heads, head_dim, pages, page_size);
  if (st != AWQ_OK) return st;
  const int64_t row = (int64_t)q_heads * head_dim;
  if (!stride_ok(ldq, row) || !stride_ok(ldy, row)) return AWQ_ERR_SHAPE;
  if (!scale_ok(scale)) return AWQ_ERR_OPTION;
  if (shared < 0 || shared % page_size != 0 || shared / page_size > width) return AWQ_ERR_OPTION;
  if (!awq::attend_fits(T, B, q_heads, kv_heads, head_dim, page_size, width, shared)) return AWQ_ERR_SHAPE;
  st = check_pointers(q, k_pages, v_pages, y);
  if (st != AWQ_OK) return st;
  st = check_workspace(workspace, workspace_bytes,
                       awq_attend_workspace_bytes(T, B, q_heads, kv_heads, head_dim, width, page_size, shared));
  if (st != AWQ_OK) return st;
  const awq::AttendArgs a{static_cast<const _Float16*>(q), ldq, q_heads, scale, nullptr, 0, shared,
                          static_cast<_Float16*>(y), ldy};
  return from_hip(awq::launch_attend(a, cache(k_pages, v_pages, nullptr, pages, kv_heads, head_dim, page_size),
                                     awq::SeqArgs{offsets, lengths, tables, width, T, B}, workspace,
                                     static_cast<hipStream_t>(stream)));
}

size_t awq_select_pages_workspace_bytes(int32_t T, int32_t kv_heads, int32_t width, int32_t count) {
  if (T < 1 || kv_heads < 1 || (int64_t)T * kv_heads >= kMaxChosen || width < 1 || count < 1) return 0;
  return awq::select_workspace_bytes(T, kv_heads, width, count);
}

int awq_select_pages(const void* q, int32_t ldq, const int32_t* offsets, const int32_t* lengths, const int32_t* tables,
                     int32_t width, int32_t T, int32_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                     const void* bounds, int32_t pages, int32_t page_size, int32_t count, int32_t first, int32_t recent,
                     int32_t* chosen, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_cache(offsets, lengths, tables, width, T, B, q_heads, kv_heads, head_dim, pages, page_size);
  if (st != AWQ_OK) return st;
  if (!stride_ok(ldq, (int64_t)q_heads * head_dim) || (int64_t)T * kv_heads >= kMaxChosen) return AWQ_ERR_SHAPE;
  if (count < 1 || first < 0 || recent < 1 || (int64_t)first + recent > count ||
      (int64_t)T * kv_heads * count >= ((int64_t)1 << 31))
    return AWQ_ERR_OPTION;
  st = check_pointers(q, bounds, bounds, bounds);
  if (st != AWQ_OK) return st;
  if (!chosen) return AWQ_ERR_NULL;
  if (!aligned4(chosen)) return AWQ_ERR_ALIGN;
  st = check_workspace(workspace, workspace_bytes, awq_select_pages_workspace_bytes(T, kv_heads, width, count));
  if (st != AWQ_OK) return st;
  const awq::SelectArgs a{static_cast<const _Float16*>(q), ldq, q_heads, count, first, recent, chosen};
  return from_hip(awq::launch_select(a, cache(nullptr, nullptr, bounds, pages, kv_heads, head_dim, page_size),
                                     awq::SeqArgs{offsets, lengths, tables, width, T, B}, workspace,
                                     static_cast<hipStream_t>(stream)));
}

size_t awq_attend_pages_workspace_bytes(int32_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                        int32_t page_size, int32_t count) {
  if (!counts_ok(T, 1, q_heads, kv_heads, 1, page_size) || !dim_known(head_dim) || count < 1) return 0;
  return awq::attend_list_workspace_bytes(T, q_heads, kv_heads, head_dim, page_size, count);
}

int awq_attend_pages(const void* q, int32_t ldq, const int32_t* offsets, const int32_t* lengths, const int32_t* tables,
                     int32_t width, int32_t T, int32_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim, float scale,
                     const int32_t* chosen, int32_t count, const void* k_pages, const void* v_pages, int32_t pages,
                     int32_t page_size, void* y, int32_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_cache(offsets, lengths, tables, width, T, B, q_heads, kv_heads, head_dim, pages, page_size);
  if (st != AWQ_OK) return st;
  const int64_t row = (int64_t)q_heads * head_dim;
  if (!stride_ok(ldq, row) || !stride_ok(ldy, row)) return AWQ_ERR_SHAPE;
  if (!scale_ok(scale)) return AWQ_ERR_OPTION;
  if (count < 1 || (int64_t)count * page_size > ((int64_t)1 << 30) ||
      (int64_t)T * kv_heads * ((q_heads / kv_heads + 15) / 16) * ((int64_t)count * page_size / 32 + 1) >= ((int64_t)1 << 30))
    return AWQ_ERR_OPTION;
  st = check_pointers(q, k_pages, v_pages, y);
  if (st != AWQ_OK) return st;
  if (!chosen) return AWQ_ERR_NULL;
  if (!aligned4(chosen)) return AWQ_ERR_ALIGN;
  st = check_workspace(workspace, workspace_bytes,
                       awq_attend_pages_workspace_bytes(T, q_heads, kv_heads, head_dim, page_size, count));
  if (st != AWQ_OK) return st;
  const awq::AttendArgs a{static_cast<const _Float16*>(q), ldq, q_heads, scale, chosen, count, 0,
                          static_cast<_Float16*>(y), ldy};
  return from_hip(awq::launch_attend(a, cache(k_pages, v_pages, nullptr, pages, kv_heads, head_dim, page_size),
                                     awq::SeqArgs{offsets, lengths, tables, width, T, B}, workspace,
                                     static_cast<hipStream_t>(stream)));
}

}  // extern "C"
