// pa_mass_tiles.cu -- the tensor-core tile launches of pa_attention_mass.
#include "pa_mass_tiles.cuh"

namespace pa {

cudaError_t launch_mass_tiles(const MassParams& p, bool weights, cudaStream_t stream) {
  // no more CTAs than there can be units (the kernel counts them from the positions)
  long long units = 0;
  for (int c = 0; c < p.n_chunks; ++c)
    units += static_cast<long long>(p.Hkv) * p.n_splits *
             (!weights ? (p.chunk_tiles[c] + 1) / 2 : p.chunk_tiles[c] > kMassLongTiles ? kMassSplitKeys / kMassLongKeys : 1);
  if (units > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (p.D == 64) return weights ? launch_mass_tile_inst<64, true>(p, units, stream) : launch_mass_tile_inst<64, false>(p, units, stream);
  return weights ? launch_mass_tile_inst<128, true>(p, units, stream) : launch_mass_tile_inst<128, false>(p, units, stream);
}

}  // namespace pa
