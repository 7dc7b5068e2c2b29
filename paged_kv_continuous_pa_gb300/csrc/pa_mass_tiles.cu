// pa_mass_tiles.cu -- the tensor-core tile launches of pa_attention_mass.
#include "pa_mass_tiles.cuh"

namespace pa {

cudaError_t launch_mass_tiles(const MassParams& p0, bool weights, cudaStream_t stream) {
  MassParams p = p0;
  const int R = kMtKeys / (p.Hq / p.Hkv);
  long long ctas = 0;
  for (int c = 0; c < p.n_chunks; ++c) {
    p.chunk_cta[c] = static_cast<int32_t>(ctas);
    const long long pairs = (p.chunk_end[c] - p.chunk_begin[c] + 2 * R - 1) / (2 * R);  // of column tiles
    ctas += weights ? static_cast<long long>(p.Hkv) * p.n_ranges : pairs * p.Hkv * p.n_splits;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  }
  p.chunk_cta[p.n_chunks] = static_cast<int32_t>(ctas);
  if (p.D == 64) return weights ? launch_mass_tile_inst<64, true>(p, ctas, stream) : launch_mass_tile_inst<64, false>(p, ctas, stream);
  return weights ? launch_mass_tile_inst<128, true>(p, ctas, stream) : launch_mass_tile_inst<128, false>(p, ctas, stream);
}

}  // namespace pa
