// linear_pair_grad.cu -- instances of linear_pair.cuh for the gradients'
// products (no epilogue but the rounding).
#include "linear_pair.cuh"

namespace gbr {

void* linear_pair_da_kernel() {
    return reinterpret_cast<void*>(&linear::linear_pair_kernel<false, false, kActNone, true>);
}
void* linear_pair_db_kernel() {
    return reinterpret_cast<void*>(&linear::linear_pair_kernel<true, true, kActNone, true>);
}

}  // namespace gbr
