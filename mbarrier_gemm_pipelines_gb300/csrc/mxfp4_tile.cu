// mxfp4_tile.cu -- instances of mxfp4_tile.cuh, one per activation.
#include "mxfp4_tile.cuh"

namespace gbr {

void* mxfp4_tile_kernel_ptr(int act) {
    using namespace mx;
    switch (act) {
        case kActRelu: return reinterpret_cast<void*>(&mxfp4_tile_kernel<kActRelu>);
        case kActGelu: return reinterpret_cast<void*>(&mxfp4_tile_kernel<kActGelu>);
        case kActGeluTanh: return reinterpret_cast<void*>(&mxfp4_tile_kernel<kActGeluTanh>);
        case kActSilu: return reinterpret_cast<void*>(&mxfp4_tile_kernel<kActSilu>);
        default: return reinterpret_cast<void*>(&mxfp4_tile_kernel<kActNone>);
    }
}

}  // namespace gbr
