// linear_tile_grad.cu -- instances of linear_tile.cuh for the gradients'
// products.
#include "linear_tile.cuh"

namespace gbr {
namespace linear {

__global__ void __launch_bounds__(kTileThreads)
    linear_tile_grads_kernel(const __grid_constant__ TileGradParams G) {
    if (blockIdx.x < G.first) tile_cta<false, false, kActNone, true>(G.da, blockIdx.x, G.cluster);
    else tile_cta<true, true, kActNone, true>(G.db, blockIdx.x - G.first, G.cluster);
}

}  // namespace linear

void* linear_tile_grads_kernel() { return reinterpret_cast<void*>(&linear::linear_tile_grads_kernel); }
void* linear_tile_da_kernel() {
    return reinterpret_cast<void*>(&linear::linear_tile_kernel<false, false, kActNone, true>);
}
void* linear_tile_db_kernel() {
    return reinterpret_cast<void*>(&linear::linear_tile_kernel<true, true, kActNone, true>);
}

}  // namespace gbr
