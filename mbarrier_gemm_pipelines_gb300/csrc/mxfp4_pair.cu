// mxfp4_pair.cu -- instances of mxfp4_pair.cuh, one per activation.
#include "mxfp4_pair.cuh"

namespace gbr {

void* mxfp4_pair_kernel_ptr(int act) {
    using namespace mx;
    switch (act) {
        case kActRelu: return reinterpret_cast<void*>(&mxfp4_pair_kernel<kActRelu>);
        case kActGelu: return reinterpret_cast<void*>(&mxfp4_pair_kernel<kActGelu>);
        case kActGeluTanh: return reinterpret_cast<void*>(&mxfp4_pair_kernel<kActGeluTanh>);
        case kActSilu: return reinterpret_cast<void*>(&mxfp4_pair_kernel<kActSilu>);
        default: return reinterpret_cast<void*>(&mxfp4_pair_kernel<kActNone>);
    }
}

}  // namespace gbr
