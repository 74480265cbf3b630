// linear_tile_forward.cu -- instances of linear_tile.cuh for C = A B with the
// full epilogue, one per activation.
#include "linear_tile.cuh"

namespace gbr {

void* linear_tile_forward_kernel(int act) {
    using namespace linear;
    switch (act) {
        case kActRelu: return reinterpret_cast<void*>(&linear_tile_kernel<true, false, kActRelu, false>);
        case kActGelu: return reinterpret_cast<void*>(&linear_tile_kernel<true, false, kActGelu, false>);
        case kActGeluTanh: return reinterpret_cast<void*>(&linear_tile_kernel<true, false, kActGeluTanh, false>);
        case kActSilu: return reinterpret_cast<void*>(&linear_tile_kernel<true, false, kActSilu, false>);
        default: return reinterpret_cast<void*>(&linear_tile_kernel<true, false, kActNone, false>);
    }
}

}  // namespace gbr
