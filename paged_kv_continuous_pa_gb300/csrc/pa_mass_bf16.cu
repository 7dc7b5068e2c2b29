// pa_mass_bf16.cu -- pa_attention_mass over bf16 pools.
#include "pa_mass.cuh"

namespace pa {

cudaError_t launch_mass_bf16(const MassParams& p, MassLaunch what, cudaStream_t stream) {
  return launch_mass_dispatch<KV_BF16>(p, what, stream);
}

}  // namespace pa
