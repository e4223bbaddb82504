// Attention of many rows (awq_attend_tiles.hpp), and of many rows of shared keys
// together with few rows per sequence (awq_attend_waves.hpp): the first is bound by
// the matrix cores, the second by HBM, and in one launch each compute unit holds a
// workgroup of either kind (61 tokens of 64 query heads after 8192: 34-36 us; one launch
// after the other, with their joins, 68 us for 46).  With heads of 256 channels a
// workgroup's ring is 128 KB, so a unit holds one at a time: the row tiles
// begin as waves end, still without the second launch (99 us, 104).
#include "awq_attend_tiles.hpp"
#include "awq_attend_waves.hpp"

namespace awq {
namespace {

template <int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attend_tiles_kernel(AttendArgs a, CacheArgs c, SeqArgs s, TileArgs x,
                                                                             Partials p) {
  __shared__ __attribute__((aligned(1024))) char ring[TileRing<D>::BYTES];
  __shared__ uint32_t strange[2];
  attend_tile<D>(a, c, s, x, p, blockIdx.x, (lds_char*)ring, strange);
}

// The first kUnits workgroups are waves on their own (kWavesOfUnit of a workgroup's four: as many as the ring has room
// for), the others row tiles of the shared keys.
template <int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attend_both_kernel(AttendArgs a, CacheArgs c, SeqArgs s,
                                                                            UnitArgs units, TileArgs x, Partials p) {
  __shared__ __attribute__((aligned(1024))) char ring[TileRing<D>::BYTES];
  __shared__ uint32_t strange[2];
  if ((int)blockIdx.x < kUnits) {
    static_assert(kWavesOfUnit * wave_ring<D>() <= TileRing<D>::BYTES, "the waves' rings fit");
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wave < kWavesOfUnit)
      attend_wave<D, 16, false>(a, c, s, units, p, blockIdx.x * kWavesOfUnit + wave, (lds_char*)ring + wave * wave_ring<D>());
  } else {
    attend_tile<D>(a, c, s, x, p, blockIdx.x - kUnits, (lds_char*)ring, strange);
  }
}

template <int D>
void launch(const AttendArgs& a, const CacheArgs& c, const SeqArgs& s, const AttendPlan& plan, const Partials& p,
            hipStream_t stream) {
  const TileArgs x = tile_args(plan, s.T, s.B, a.q_heads, c.heads, c.dim);
  const unsigned grid = (unsigned)tile_workgroups(x, c.heads);
  if (plan.both())
    hipLaunchKernelGGL((attend_both_kernel<D>), dim3(kUnits + grid), dim3(256), 0, stream, a, c, s, unit_args(a, c, plan), x,
                       p);
  else
    hipLaunchKernelGGL((attend_tiles_kernel<D>), dim3(grid), dim3(256), 0, stream, a, c, s, x, p);
}

}  // namespace

hipError_t launch_attend_tiles(const AttendArgs& a, const CacheArgs& c, const SeqArgs& s, const AttendPlan& plan,
                               const Partials& p, hipStream_t stream) {
  if (c.dim == 64) launch<64>(a, c, s, plan, p, stream);
  else if (c.dim == 96) launch<96>(a, c, s, plan, p, stream);
  else if (c.dim == 128) launch<128>(a, c, s, plan, p, stream);
  else launch<256>(a, c, s, plan, p, stream);
  return hipGetLastError();
}

}  // namespace awq
