// pa_mass_f32.cu -- pa_attention_mass over f32 pools.
#include "pa_mass.cuh"

namespace pa {

cudaError_t launch_mass_f32(const MassParams& p, MassLaunch what, cudaStream_t stream) {
  return launch_mass_dispatch<KV_F32>(p, what, stream);
}

}  // namespace pa
