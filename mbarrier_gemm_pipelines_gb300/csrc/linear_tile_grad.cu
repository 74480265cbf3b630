// linear_tile_grad.cu -- instances of linear_tile.cuh for the gradients'
// products.
#include "linear_tile.cuh"

namespace gbr {

void* linear_tile_da_kernel() {
    return reinterpret_cast<void*>(&linear::linear_tile_kernel<false, false, kActNone, true>);
}
void* linear_tile_db_kernel() {
    return reinterpret_cast<void*>(&linear::linear_tile_kernel<true, true, kActNone, true>);
}

}  // namespace gbr
