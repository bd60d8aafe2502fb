// csa_attn_prefix.cu -- the tensor-core kernels of the attention behind shared prefixes (csa_attn_tile.cuh);
// their plan, and what is done where they do not run, stand in csa_attn.cu.
#include "csa_attn_tile.cuh"

namespace csa {

TileKernels prefix_tile_kernels(int nc, int source, int format) { return tile_kernels<true>(nc, source, format); }

}  // namespace csa
