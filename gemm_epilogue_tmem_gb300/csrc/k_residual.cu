// Instances: RESIDUAL (out = act(acc + bias) + residual).
#include "dispatch.cuh"

namespace gf {

cudaError_t launch_residual(const LaunchArgs& a) { return launch_epi<EPI_RESIDUAL>(a); }

}  // namespace gf
