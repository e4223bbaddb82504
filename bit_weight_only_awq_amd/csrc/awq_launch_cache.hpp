// Host-side launchers of the operators on a paged cache of keys and values.
// Arguments are validated by the C ABI layer; each launcher returns
// hipGetLastError() after enqueueing its kernels on `stream`.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace awq {

// B sequences with T rows of new tokens among them.
struct SeqArgs {
  const int* offsets;  // [B + 1]: sequence b's rows are offsets[b] .. offsets[b + 1] - 1
  const int* lengths;  // [B]: its tokens, the new ones among them
  const int* tables;   // [B][width]: its pages
  int width, T, B;
};

// Pages of S = 1 << shift tokens, [pages][heads][S][dim] each for keys and values.
struct CacheArgs {
  _Float16* k;
  _Float16* v;
  _Float16* bounds;  // [pages][heads][2][dim]: each page's lowest and highest key, or NULL
  int pages, heads, dim, shift;
};

struct AppendArgs {
  const _Float16* x;  // rows of q_heads + 2 heads vectors of dim: queries, keys, values
  int64_t ldx;
  int q_heads;
  const float* inv_freq;  // [rotary / 2]
  int rotary;
  bool interleaved;
  const int* positions;  // [T][axes], or NULL: the token's place in its sequence
  int axes;
  const int* axis;  // [rotary / 2], or NULL: axis 0
  _Float16* q;
  int64_t ldq;
};
hipError_t launch_append(const AppendArgs& a, const CacheArgs& c, const SeqArgs& s, hipStream_t stream);

struct AttendArgs {
  const _Float16* q;  // row t: q_heads vectors of dim
  int64_t ldq;
  int q_heads;
  float scale;
  const int* list;  // [T][heads][count]: pages of the token's sequence, negative: none; or NULL: all of them
  int count;
  int shared;  // keys that every sequence begins with, read through the table of the first that has rows
  _Float16* y;
  int64_t ldy;
};
// Whether the launch has less than 2^32 threads (with shared keys beside a row tile for nearly each of 2^24 rows it has not).
bool attend_fits(int T, int B, int q_heads, int kv_heads, int dim, int page_size, int width, int shared);
size_t attend_workspace_bytes(int T, int B, int q_heads, int kv_heads, int dim, int page_size, int width, int shared);
size_t attend_list_workspace_bytes(int T, int q_heads, int kv_heads, int dim, int page_size, int count);
hipError_t launch_attend(const AttendArgs& a, const CacheArgs& c, const SeqArgs& s, void* workspace, hipStream_t stream);

struct SelectArgs {
  const _Float16* q;
  int64_t ldq;
  int q_heads, count, first, recent;
  int* pages;  // [T][heads][count]
};
size_t select_workspace_bytes(int T, int kv_heads, int width, int count);
hipError_t launch_select(const SelectArgs& a, const CacheArgs& c, const SeqArgs& s, void* workspace, hipStream_t stream);

}  // namespace awq
