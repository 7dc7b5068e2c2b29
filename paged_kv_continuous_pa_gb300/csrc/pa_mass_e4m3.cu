// pa_mass_e4m3.cu -- pa_attention_mass over e4m3 pools.
#include "pa_mass.cuh"

namespace pa {

cudaError_t launch_mass_e4m3(const MassParams& p, MassLaunch what, cudaStream_t stream) {
  return launch_mass_dispatch<KV_E4M3>(p, what, stream);
}

}  // namespace pa
