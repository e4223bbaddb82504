// Attention of few rows per sequence on its own: a workgroup is one wave
// (awq_attend_waves.hpp), so nothing waits for a barrier.
#include "awq_attend_waves.hpp"

namespace awq {
namespace {

template <int D, int R, bool LIST>
__global__ __launch_bounds__(64, D == 256 ? 1 : 2) void attend_waves_kernel(AttendArgs a, CacheArgs c, SeqArgs s,
                                                                            UnitArgs units, Partials p) {
  __shared__ __attribute__((aligned(1024))) char ring[wave_ring<D>()];
  attend_wave<D, R, LIST>(a, c, s, units, p, blockIdx.x, (lds_char*)ring);
}

template <int D, int R>
void launch_as(const AttendArgs& a, const CacheArgs& c, const SeqArgs& s, const AttendPlan& plan, const Partials& p,
               const UnitArgs& u, hipStream_t stream) {
  if (a.list) hipLaunchKernelGGL((attend_waves_kernel<D, R, true>), dim3(kWaves), dim3(64), 0, stream, a, c, s, u, p);
  else hipLaunchKernelGGL((attend_waves_kernel<D, R, false>), dim3(kWaves), dim3(64), 0, stream, a, c, s, u, p);
}

template <int D>
void launch(const AttendArgs& a, const CacheArgs& c, const SeqArgs& s, const AttendPlan& plan, const Partials& p,
            const UnitArgs& u, hipStream_t stream) {
  if (plan.rows == 16) launch_as<D, 16>(a, c, s, plan, p, u, stream);
  else launch_as<D, 32>(a, c, s, plan, p, u, stream);
}

}  // namespace

hipError_t launch_attend_waves(const AttendArgs& a, const CacheArgs& c, const SeqArgs& s, const AttendPlan& plan,
                               const Partials& p, hipStream_t stream) {
  const UnitArgs u = unit_args(a, c, plan);
  if (c.dim == 64) launch<64>(a, c, s, plan, p, u, stream);
  else if (c.dim == 96) launch<96>(a, c, s, plan, p, u, stream);
  else if (c.dim == 128) launch<128>(a, c, s, plan, p, u, stream);
  else launch<256>(a, c, s, plan, p, u, stream);
  return hipGetLastError();
}

}  // namespace awq
